"""Thin Python binding of libmoe_lora.so (include/moe_lora.h).

Argument marshalling only: each function checks tensor dtypes / devices,
passes raw pointers and sizes to the C ABI of the same name and raises
MoeLoraError on a non-zero status.  Every step of the computation runs in
the library's CUDA kernels; there is no other implementation to fall back to,
so a missing library is an error.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
import warnings

import torch

from . import build as _build

MOE_LORA_OK = 0
ALIGN_AUTO, ALIGN_SMEM, ALIGN_GLOBAL, ALIGN_CLUSTER = 0, 1, 2, 3
ROUTE_SOFTMAX, ROUTE_SIGMOID = 0, 1
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4
PATH_AUTO, PATH_CUDA_CORE, PATH_TCGEN05, PATH_CUDA_CORE_CLUSTER, PATH_CUDA_CORE_STREAM = 0, 1, 2, 3, 4
DEVERR_EXPERT_ID, DEVERR_LORA_ID, DEVERR_CAPACITY, DEVERR_PAIR_ID, DEVERR_TIMEOUT = 1, 2, 4, 8, 16

_lib = None
_fast = None     # fastcall's functions, or a stand-in
_lock = threading.Lock()


class MoeLoraError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (what, status_string(status), status))


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libmoe_lora.so (building it with nvcc if it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            if not os.path.exists(path):
                raise RuntimeError("libmoe_lora.so is missing: " + path)
            L = ctypes.CDLL(path)
            I, P, S = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
            L.moe_lora_version.restype = I
            L.moe_lora_version.argtypes = []
            L.moe_lora_status_string.restype = ctypes.c_char_p
            L.moe_lora_status_string.argtypes = [I]
            L.moe_lora_max_num_tokens_padded.restype = I
            L.moe_lora_max_num_tokens_padded.argtypes = [I, I, I, I]
            L.moe_lora_max_num_m_blocks.restype = I
            L.moe_lora_max_num_m_blocks.argtypes = [I, I, I, I]
            L.moe_lora_align_resolve_variant.restype = I
            L.moe_lora_align_resolve_variant.argtypes = [I, I, I, I]
            L.moe_lora_align_workspace_bytes.restype = S
            L.moe_lora_align_workspace_bytes.argtypes = [I, I, I, I, I, I]
            L.moe_lora_align.restype = I
            L.moe_lora_align.argtypes = [P, P, P, P, I, I, I, I, I, I, P, P, P, I, I, P, S, I, P, P]
            L.moe_lora_align_static_workspace.restype = I
            L.moe_lora_align_static_workspace.argtypes = [P, P, P, P, I, I, I, I, I, I, P, P, P, I, I, P, P]
            L.moe_lora_fused_shrink_expand.restype = I
            L.moe_lora_fused_shrink_expand.argtypes = [P, P, P, P, P, P, P, P, P,
                                                       I, I, I, I, I, I, I, I, I, I, I, I, I, P, P]
            L.moe_lora_fused_shrink_expand_ex.restype = I
            L.moe_lora_fused_shrink_expand_ex.argtypes = [P, I, ctypes.POINTER(P), ctypes.POINTER(P), I, P, I, I, P,
                                                          P, P, P, P, P,
                                                          I, I, I, I, I, I, I, I, I, I, I, I, I, P, P]
            L.moe_align_block_size.restype = I
            L.moe_align_block_size.argtypes = [P, I, I, I, I, P, P, P, I, I, P, S, I, P, P]
            L.moe_lora_fused_shrink_expand_naive.restype = I
            L.moe_lora_fused_shrink_expand_naive.argtypes = [P, I, ctypes.POINTER(P), ctypes.POINTER(P), I, P, I, I,
                                                             P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, P,
                                                             P]
            L.moe_lora_test_withheld_copy.restype = I
            L.moe_lora_test_withheld_copy.argtypes = [P, I, ctypes.POINTER(P), ctypes.POINTER(P), I, P, I, I, P, P,
                                                      P, P, P, I, I, I, I, I, I, I, I, I, ctypes.c_ulonglong, P, P]
            L.moe_lora_fused_plan.restype = I
            L.moe_lora_fused_plan.argtypes = [I] * 12 + [P]
            L.moe_lora_fused_resolve_path.restype = I
            L.moe_lora_fused_resolve_path.argtypes = [I] * 10
            L.moe_lora_fused_naive_resolve_path.restype = I
            L.moe_lora_fused_naive_resolve_path.argtypes = [I] * 9
            Q, F = ctypes.c_longlong, ctypes.c_float
            L.moe_add_rms_norm_fp8.restype = I
            L.moe_add_rms_norm_fp8.argtypes = [P, Q, Q, I, P, Q, P, F, P, Q, P, Q, P, Q, P, I, I, P]
            L.moe_silu_mul_fp8.restype = I
            L.moe_silu_mul_fp8.argtypes = [P, Q, P, Q, P, Q, P, I, I, P]
            L.moe_fp8_matmul.restype = I
            L.moe_fp8_matmul.argtypes = [P, Q, P, P, Q, P, P, Q, I, I, I, P, P]
            L.moe_fp8_grouped_matmul.restype = I
            L.moe_fp8_grouped_matmul.argtypes = [P, I, Q, P, P, Q, P, P, Q, P, P, P, P, I, I, I, I, I, I, I, I, P, S, P, P]
            L.moe_fp8_grouped_workspace_bytes.restype = S
            L.moe_fp8_grouped_workspace_bytes.argtypes = [I, I, I, I, I, I]
            L.moe_fp8_grouped_matmul_naive.restype = I
            L.moe_fp8_grouped_matmul_naive.argtypes = [P, I, Q, P, P, Q, P, P, Q, P, P, I, I, I, I, I, P, P]
            L.moe_route.restype = I
            L.moe_route.argtypes = [P, I, Q, P, I, I, F, I, I, I, P, P, I, I, I, P]
            L.moe_bf16_matmul.restype = I
            L.moe_bf16_matmul.argtypes = [P, Q, P, Q, P, I, P, Q, P, Q, I, I, I, I, I, P, P]
            L.moe_bf16_grouped_matmul.restype = I
            L.moe_bf16_grouped_matmul.argtypes = [P, I, Q, P, Q, P, I, P, Q, I, P, P, P, P, I, I, I, I, I, I, I, I, P, S,
                                                  P, P]
            L.moe_bf16_grouped_workspace_bytes.restype = S
            L.moe_bf16_grouped_workspace_bytes.argtypes = [I, I, I, I, I, I]
            L.moe_bf16_grouped_matmul_naive.restype = I
            L.moe_bf16_grouped_matmul_naive.argtypes = [P, I, Q, P, Q, P, I, P, Q, I, P, P, I, I, I, I, I, P, P]
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_lora_status_string(int(status)).decode()


def max_num_tokens_padded(M: int, topk: int, num_experts: int, block_size: int) -> int:
    return lib().moe_lora_max_num_tokens_padded(M, topk, num_experts, block_size)


def max_num_m_blocks(M: int, topk: int, num_experts: int, block_size: int) -> int:
    return lib().moe_lora_max_num_m_blocks(M, topk, num_experts, block_size)


def align_resolve_variant(M, topk, num_experts, variant=ALIGN_AUTO) -> int:
    """The align variant a call with these sizes runs (ALIGN_SMEM, ALIGN_GLOBAL
    or ALIGN_CLUSTER)."""
    v = lib().moe_lora_align_resolve_variant(M, topk, num_experts, variant)
    if v < 0:
        raise MoeLoraError(-v, "moe_lora_align_resolve_variant")
    return v


def align_workspace_bytes(M, topk, num_experts, num_active_loras, block_size, variant=ALIGN_AUTO) -> int:
    return lib().moe_lora_align_workspace_bytes(M, topk, num_experts, num_active_loras, block_size, variant)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(status, what):
    if status != MOE_LORA_OK:
        raise MoeLoraError(status, what)


def moe_lora_align(topk_ids, token_lora_mapping, lora_ids, num_experts, max_loras, block_size,
                   sorted_token_ids, expert_ids, num_tokens_post_padded, adapter_enabled=None,
                   workspace=None, variant=ALIGN_AUTO, err_flag=None, stream=None):
    """moe_lora_align on device tensors; outputs are written in place."""
    M, topk = topk_ids.shape
    nact = lora_ids.numel()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().moe_lora_align(
        _ptr(topk_ids, torch.int32, "topk_ids"), _ptr(token_lora_mapping, torch.int32, "token_lora_mapping"),
        _ptr(lora_ids, torch.int32, "lora_ids"), _ptr(adapter_enabled, torch.int32, "adapter_enabled"),
        M, topk, num_experts, max_loras, nact, block_size,
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"), _ptr(expert_ids, torch.int32, "expert_ids"),
        _ptr(num_tokens_post_padded, torch.int32, "num_tokens_post_padded"),
        sorted_token_ids.shape[-1], expert_ids.shape[-1],
        _ptr(workspace, None, "workspace"), ws_bytes, variant,
        _ptr(err_flag, torch.int32, "err_flag"), _stream(stream))
    _check(st, "moe_lora_align")


STATIC_WORKSPACE_BYTES = 4 << 20


def moe_align_block_size(topk_ids, num_experts, block_size, sorted_token_ids, expert_ids, num_tokens_post_padded,
                         workspace=None, variant=ALIGN_AUTO, err_flag=None, stream=None):
    """The plain (non-LoRA) MoE align on device tensors: outputs are
    sorted_token_ids [cap], expert_ids [capb], num_tokens_post_padded [1]."""
    M, topk = topk_ids.shape
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().moe_align_block_size(
        _ptr(topk_ids, torch.int32, "topk_ids"), M, topk, num_experts, block_size,
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"), _ptr(expert_ids, torch.int32, "expert_ids"),
        _ptr(num_tokens_post_padded, torch.int32, "num_tokens_post_padded"),
        sorted_token_ids.numel(), expert_ids.numel(), _ptr(workspace, name="workspace"), nbytes, variant,
        _ptr(err_flag, torch.int32, "err_flag"), _stream(stream))
    _check(st, "moe_align_block_size")


def moe_lora_align_static_workspace(topk_ids, token_lora_mapping, lora_ids, num_experts, max_loras, block_size,
                                    sorted_token_ids, expert_ids, num_tokens_post_padded, adapter_enabled=None,
                                    err_flag=None, stream=None):
    """moe_lora_align (global variant) on the library's built-in scratch buffer,
    for callers that cannot allocate device memory; see include/moe_lora.h."""
    M, topk = topk_ids.shape
    st = lib().moe_lora_align_static_workspace(
        _ptr(topk_ids, torch.int32, "topk_ids"), _ptr(token_lora_mapping, torch.int32, "token_lora_mapping"),
        _ptr(lora_ids, torch.int32, "lora_ids"), _ptr(adapter_enabled, torch.int32, "adapter_enabled"),
        M, topk, num_experts, max_loras, lora_ids.numel(), block_size,
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"), _ptr(expert_ids, torch.int32, "expert_ids"),
        _ptr(num_tokens_post_padded, torch.int32, "num_tokens_post_padded"),
        sorted_token_ids.shape[-1], expert_ids.shape[-1],
        _ptr(err_flag, torch.int32, "err_flag"), _stream(stream))
    _check(st, "moe_lora_align_static_workspace")


def moe_lora_fused_shrink_expand(x, lora_a, lora_b, y, sorted_token_ids, expert_ids, num_tokens_post_padded,
                                 lora_ids, topk, block_size, add_inputs=True, adapter_enabled=None,
                                 path=PATH_AUTO, err_flag=None, stream=None):
    """moe_lora_fused_shrink_expand on device tensors; y is updated in place."""
    M, K = x.shape
    L, E, r, K2 = lora_a.shape
    N = lora_b.shape[2]
    if K2 != K or tuple(lora_b.shape) != (L, E, N, r) or y.numel() != M * topk * N:
        raise ValueError("inconsistent shapes")
    bf = torch.bfloat16
    st = lib().moe_lora_fused_shrink_expand(
        _ptr(x, bf, "x"), _ptr(lora_a, bf, "lora_a"), _ptr(lora_b, bf, "lora_b"), _ptr(y, bf, "y"),
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"), _ptr(expert_ids, torch.int32, "expert_ids"),
        _ptr(num_tokens_post_padded, torch.int32, "num_tokens_post_padded"),
        _ptr(lora_ids, torch.int32, "lora_ids"), _ptr(adapter_enabled, torch.int32, "adapter_enabled"),
        M, topk, E, K, N, r, L, lora_ids.numel(), block_size,
        sorted_token_ids.shape[-1], expert_ids.shape[-1], int(bool(add_inputs)), path,
        _ptr(err_flag, torch.int32, "err_flag"), _stream(stream))
    _check(st, "moe_lora_fused_shrink_expand")


def fused_naive_resolve_path(M, topk, num_experts, K, N, rank, num_active_loras, num_slices=1, path=PATH_AUTO) -> int:
    """The kernel a naive-assignment call with these sizes runs
    (PATH_CUDA_CORE_CLUSTER or PATH_CUDA_CORE_STREAM)."""
    v = lib().moe_lora_fused_naive_resolve_path(M, topk, num_experts, K, N, rank, num_active_loras, num_slices, path)
    if v < 0:
        raise MoeLoraError(-v, "moe_lora_fused_naive_resolve_path")
    return v


def fused_resolve_path(M, topk, num_experts, K, N, rank, num_active_loras, block_size, num_slices=1,
                       path=PATH_AUTO) -> int:
    """The kernel a fused call with these sizes runs (PATH_TCGEN05,
    PATH_CUDA_CORE_CLUSTER or PATH_CUDA_CORE_STREAM)."""
    v = lib().moe_lora_fused_resolve_path(M, topk, num_experts, K, N, rank, num_active_loras, block_size,
                                          num_slices, path)
    if v < 0:
        raise MoeLoraError(-v, "moe_lora_fused_resolve_path")
    return v


PLAN_FIELDS = ("kernel", "grid", "threads", "smem_bytes", "s_sh", "lag", "s_ex", "t_bufs", "tmem_cols", "cluster",
               "pairs_per_group")


def fused_plan(M, topk, num_experts, K, N, rank, num_active_loras, block_size, num_slices=1, path=PATH_AUTO,
               sm_count=152, max_smem_per_block=232448) -> dict:
    """The launch plan a plain fused call would use on a device with these
    properties (host arithmetic only)."""
    out = (ctypes.c_int32 * len(PLAN_FIELDS))()
    st = lib().moe_lora_fused_plan(M, topk, num_experts, K, N, rank, num_active_loras, block_size, num_slices, path,
                                   sm_count, max_smem_per_block, ctypes.cast(out, ctypes.c_void_p))
    _check(st, "moe_lora_fused_plan")
    return dict(zip(PLAN_FIELDS, list(out)))


def moe_lora_fused_shrink_expand_ex(x, lora_a, lora_b, y, sorted_token_ids, expert_ids, num_tokens_post_padded,
                                    lora_ids, topk, block_size, add_inputs=True, adapter_enabled=None,
                                    topk_weights=None, x_per_pair=False, y_offset=0,
                                    path=PATH_AUTO, err_flag=None, stream=None):
    """moe_lora_fused_shrink_expand_ex on device tensors; y is updated in place.

    lora_a / lora_b: a tensor (one slice) or a list of per-slice tensors
    ([L, E, r, K] / [L, E, N, r]).  x: [M, K], or [M*topk, K] with x_per_pair.
    y: [M, topk, ldy]; slice s writes columns y_offset + s*N .. + N.
    topk_weights: float32 [M, topk] or None."""
    if isinstance(lora_a, torch.Tensor):
        lora_a, lora_b = [lora_a], [lora_b]
    S = len(lora_a)
    if S < 1 or len(lora_b) != S:
        raise ValueError("lora_a and lora_b need the same number of slices")
    L, E, r, K = lora_a[0].shape
    N = lora_b[0].shape[2]
    for a, b in zip(lora_a, lora_b):
        if tuple(a.shape) != (L, E, r, K) or tuple(b.shape) != (L, E, N, r):
            raise ValueError("inconsistent slice shapes")
    if y.dim() != 3:
        raise ValueError("y must be [M, topk, ldy]")
    M = y.shape[0]
    ldy = y.shape[2]
    if y.shape[1] != topk or tuple(x.shape) != ((M * topk if x_per_pair else M), K):
        raise ValueError("inconsistent shapes")
    if topk_weights is not None and topk_weights.numel() != M * topk:
        raise ValueError("topk_weights must be [M, topk]")
    bf = torch.bfloat16
    a_ptrs = (ctypes.c_void_p * S)(*[_ptr(a, bf, "lora_a") for a in lora_a])
    b_ptrs = (ctypes.c_void_p * S)(*[_ptr(b, bf, "lora_b") for b in lora_b])
    st = lib().moe_lora_fused_shrink_expand_ex(
        _ptr(x, bf, "x"), int(bool(x_per_pair)), a_ptrs, b_ptrs, S, _ptr(y, bf, "y"), ldy, y_offset,
        _ptr(topk_weights, torch.float32, "topk_weights"),
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"), _ptr(expert_ids, torch.int32, "expert_ids"),
        _ptr(num_tokens_post_padded, torch.int32, "num_tokens_post_padded"),
        _ptr(lora_ids, torch.int32, "lora_ids"), _ptr(adapter_enabled, torch.int32, "adapter_enabled"),
        M, topk, E, K, N, r, L, lora_ids.numel(), block_size,
        sorted_token_ids.shape[-1], expert_ids.shape[-1], int(bool(add_inputs)), path,
        _ptr(err_flag, torch.int32, "err_flag"), _stream(stream))
    _check(st, "moe_lora_fused_shrink_expand_ex")


def moe_lora_fused_shrink_expand_naive(x, lora_a, lora_b, y, topk_ids, token_lora_mapping, lora_ids, max_loras,
                                       add_inputs=True, adapter_enabled=None, topk_weights=None, x_per_pair=False,
                                       y_offset=0, path=PATH_AUTO, err_flag=None, stream=None):
    """moe_lora_fused_shrink_expand_naive (no align: one work item per pair) on
    device tensors; y [M, topk, ldy] is updated in place.  lora_a / lora_b: a
    tensor or a list of per-slice tensors.  path: PATH_AUTO, PATH_CUDA_CORE,
    PATH_CUDA_CORE_CLUSTER or PATH_CUDA_CORE_STREAM."""
    if isinstance(lora_a, torch.Tensor):
        lora_a, lora_b = [lora_a], [lora_b]
    S = len(lora_a)
    if S < 1 or len(lora_b) != S:
        raise ValueError("lora_a and lora_b need the same number of slices")
    L, E, r, K = lora_a[0].shape
    N = lora_b[0].shape[2]
    for a, b in zip(lora_a, lora_b):
        if tuple(a.shape) != (L, E, r, K) or tuple(b.shape) != (L, E, N, r):
            raise ValueError("inconsistent slice shapes")
    M, topk = topk_ids.shape
    if y.dim() != 3 or y.shape[0] != M or y.shape[1] != topk:
        raise ValueError("y must be [M, topk, ldy]")
    if tuple(x.shape) != ((M * topk if x_per_pair else M), K) or token_lora_mapping.numel() != M:
        raise ValueError("inconsistent shapes")
    if topk_weights is not None and topk_weights.numel() != M * topk:
        raise ValueError("topk_weights must be [M, topk]")
    if max_loras != L:
        raise ValueError("max_loras must equal the adapters' first dimension")
    bf = torch.bfloat16
    a_ptrs = (ctypes.c_void_p * S)(*[_ptr(a, bf, "lora_a") for a in lora_a])
    b_ptrs = (ctypes.c_void_p * S)(*[_ptr(b, bf, "lora_b") for b in lora_b])
    st = lib().moe_lora_fused_shrink_expand_naive(
        _ptr(x, bf, "x"), int(bool(x_per_pair)), a_ptrs, b_ptrs, S, _ptr(y, bf, "y"), y.shape[2], y_offset,
        _ptr(topk_weights, torch.float32, "topk_weights"), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(token_lora_mapping, torch.int32, "token_lora_mapping"), _ptr(lora_ids, torch.int32, "lora_ids"),
        _ptr(adapter_enabled, torch.int32, "adapter_enabled"), M, topk, E, K, N, r, L, lora_ids.numel(),
        int(bool(add_inputs)), int(path), _ptr(err_flag, torch.int32, "err_flag"), _stream(stream))
    _check(st, "moe_lora_fused_shrink_expand_naive")


def moe_lora_test_withheld_copy(x, lora_a, lora_b, y, topk_ids, token_lora_mapping, lora_ids, max_loras,
                                wait_limit_ns, add_inputs=True, err_flag=None, stream=None):
    """moe_lora_test_withheld_copy (a test of the bounded waits): the naive call
    with every CTA's B-slice copy withheld and its wait limited to
    wait_limit_ns; y [M, topk, N], one slice."""
    if isinstance(lora_a, torch.Tensor):
        lora_a, lora_b = [lora_a], [lora_b]
    S = len(lora_a)
    L, E, r, K = lora_a[0].shape
    N = lora_b[0].shape[2]
    M, topk = topk_ids.shape
    bf = torch.bfloat16
    a_ptrs = (ctypes.c_void_p * S)(*[_ptr(a, bf, "lora_a") for a in lora_a])
    b_ptrs = (ctypes.c_void_p * S)(*[_ptr(b, bf, "lora_b") for b in lora_b])
    st = lib().moe_lora_test_withheld_copy(
        _ptr(x, bf, "x"), 0, a_ptrs, b_ptrs, S, _ptr(y, bf, "y"), y.shape[2], 0, None,
        _ptr(topk_ids, torch.int32, "topk_ids"), _ptr(token_lora_mapping, torch.int32, "token_lora_mapping"),
        _ptr(lora_ids, torch.int32, "lora_ids"), None, M, topk, E, K, N, r, L, lora_ids.numel(),
        int(bool(add_inputs)), int(wait_limit_ns), _ptr(err_flag, torch.int32, "err_flag"), _stream(stream))
    _check(st, "moe_lora_test_withheld_copy")


class _NoFast:
    """Stands in for fastcall where it was not built or does not load: every call goes through ctypes."""

    @staticmethod
    def norm(*args):
        return None

    act = matmul = grouped = naive = route = matmul16 = grouped16 = naive16 = norm


def _load_fast():
    """fastcall's functions (a compiled module): they take the common case of the
    serving operators' calls (ordinary tensors on the current device, its current
    stream) and return None for any other, which the functions below treat."""
    global _fast
    L = lib()
    with _lock:
        if _fast is None:
            fast = None
            if os.path.exists(_build.FASTCALL):
                try:
                    spec = importlib.util.spec_from_file_location("fastcall", _build.FASTCALL)
                    fast = importlib.util.module_from_spec(spec)
                    spec.loader.exec_module(fast)
                except ImportError as e:
                    warnings.warn("the serving operators' calls go through ctypes: %s" % e)
                    fast = None
            if fast is not None:
                fast.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
                    L.moe_add_rms_norm_fp8, L.moe_silu_mul_fp8, L.moe_fp8_matmul, L.moe_fp8_grouped_matmul,
                    L.moe_fp8_grouped_matmul_naive, L.moe_fp8_grouped_workspace_bytes)])
                fast.bind16(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
                    L.moe_route, L.moe_bf16_matmul, L.moe_bf16_grouped_matmul, L.moe_bf16_grouped_matmul_naive,
                    L.moe_bf16_grouped_workspace_bytes)])
                _fast = fast
            else:
                _fast = _NoFast
    return _fast


FP8_GROUP = 128   # columns that share a scale

_BF16, _F8, _F32, _I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32


def fp8_groups(columns: int) -> int:
    """Scales of a row of `columns` 8-bit values."""
    return -(-columns // FP8_GROUP)


def _dense(t, dtype, name, numel=None):
    """Address of a contiguous CUDA tensor (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if numel is not None and t.numel() != numel:
        raise ValueError("%s must have %d elements, got shape %s" % (name, numel, tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows(t, dtype, name, rows, columns):
    """Address and leading dimension of the rows of a CUDA tensor: its last
    dimension dense, the ones before it as if they were one of `rows`."""
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    shape = t.shape
    if shape[-1] != columns or t.numel() != rows * columns:
        raise ValueError("%s: inconsistent shapes: [.., %d, %d] wanted, got %s" % (name, rows, columns, tuple(shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if rows == 1:            # one row: any leading dimension will do
        if columns > 1 and t.stride(-1) != 1:
            raise ValueError("%s must have dense rows" % name)
        return t.data_ptr(), -(-columns // 16) * 16
    if t.is_contiguous():
        return t.data_ptr(), columns
    stride = t.stride()
    if len(shape) < 2 or (stride[-1] != 1 and columns > 1):
        raise ValueError("%s must have dense rows, got shape %s, strides %s" % (name, tuple(shape), stride))
    # the dimensions of one row each say nothing
    dims = [(n, st) for n, st in zip(shape[:-1], stride[:-1]) if n > 1]
    step = ld = dims[-1][1]
    for n, st in reversed(dims):
        if st != step:
            raise ValueError("%s's rows must be evenly spaced, got shape %s, strides %s" % (name, tuple(shape), stride))
        step *= n
    return t.data_ptr(), ld


_raw_current_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _raw_stream(stream, t):
    if stream is None:
        if _raw_current_stream is None:
            return torch.cuda.current_stream(t.device).cuda_stream
        return _raw_current_stream(t.get_device())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _check_device(stream, *tensors):
    """The library works on the current device, and the stream is taken from a tensor's: all of a call's tensors, and a
    stream that the caller names, must be there."""
    here = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError("a tensor on cuda:%d, with cuda:%d as the current device" % (t.get_device(), here))
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != here:
        raise ValueError("a stream of cuda:%d, with cuda:%d as the current device" % (stream.device.index, here))


def moe_add_rms_norm_fp8(x, weight, q, scales, residual=None, residual_out=None, normed=None, eps=1e-6, stream=None):
    """Residual addition and root-mean-square norm with an 8-bit output; see
    include/moe_lora.h.

    x: bf16 [M, H], or [M, parts, H] (a token's rows, summed).  residual,
    residual_out, normed: bf16 [M, H] or None.  q: float8_e4m3fn [M, H];
    scales: float32 [M, ceil(H / 128)].  Rows may be strided."""
    if stream is None:
        st = (_fast or _load_fast()).norm(x, weight, q, scales, residual, residual_out, normed, eps)
        if st is not None:
            return _check(st, "moe_add_rms_norm_fp8")
    shape = x.shape
    M, H = shape[0], shape[-1]
    parts, ld_part = 1, 0
    if len(shape) == 3:
        parts = shape[1]
        if x.dtype is not _BF16 or not x.is_cuda:
            raise TypeError("x must be a bfloat16 CUDA tensor")
        ldx, ld_part, one = x.stride()
        if one != 1 and H > 1:
            raise ValueError("x must have dense rows")
        if parts == 1:
            ld_part = 0
        if M == 1:
            ldx = max(ldx, H)
        px = x.data_ptr()
    else:
        px, ldx = _rows(x, _BF16, "x", M, H)
    pr, ldr = (None, 0) if residual is None else _rows(residual, _BF16, "residual", M, H)
    po, ldo = (None, 0) if residual_out is None else _rows(residual_out, _BF16, "residual_out", M, H)
    pn, ldn = (None, 0) if normed is None else _rows(normed, _BF16, "normed", M, H)
    pq, ldq = _rows(q, _F8, "q", M, H)
    pw, ps = _dense(weight, _BF16, "weight", H), _dense(scales, _F32, "scales", M * -(-H // FP8_GROUP))
    _check_device(stream, x, weight, q, scales, residual, residual_out, normed)
    _check((_lib or lib()).moe_add_rms_norm_fp8(px, ldx, ld_part, parts, pr, ldr, pw, eps, po, ldo, pn, ldn, pq, ldq, ps,
                                                M, H, _raw_stream(stream, q)), "moe_add_rms_norm_fp8")


def moe_silu_mul_fp8(x, q, scales, act=None, stream=None):
    """silu(gate) * up with an 8-bit output; see include/moe_lora.h.

    x: bf16 [..., 2*I], gate then up.  q: float8_e4m3fn [..., I]; scales:
    float32 [..., ceil(I / 128)]; act: bf16 [..., I] or None.  Rows may be
    strided, evenly."""
    if stream is None:
        st = (_fast or _load_fast()).act(x, q, scales, act)
        if st is not None:
            return _check(st, "moe_silu_mul_fp8")
    I = q.shape[-1]
    rows = q.numel() // I if I else 0
    px, ldx = _rows(x, _BF16, "x", rows, 2 * I)
    pa, lda = (None, 0) if act is None else _rows(act, _BF16, "act", rows, I)
    pq, ldq = _rows(q, _F8, "q", rows, I)
    ps = _dense(scales, _F32, "scales", rows * -(-I // FP8_GROUP))
    _check_device(stream, x, q, scales, act)
    _check((_lib or lib()).moe_silu_mul_fp8(px, ldx, pa, lda, pq, ldq, ps, rows, I, _raw_stream(stream, q)),
           "moe_silu_mul_fp8")


def moe_fp8_matmul(x, x_scales, w, w_scales, y, err_flag=None, stream=None):
    """y = x @ w.T, 8-bit operands with a scale for each block of 128; see
    include/moe_lora.h.

    x: float8_e4m3fn [M, K], x_scales: float32 [M, ceil(K / 128)]; w:
    float8_e4m3fn [N, K], w_scales: float32 [ceil(N / 128), ceil(K / 128)]; y:
    bf16 [M, N].  Rows of x, w and y may be strided (x, w: by multiples of 16)."""
    if stream is None:
        st = (_fast or _load_fast()).matmul(x, x_scales, w, w_scales, y, err_flag)
        if st is not None:
            return _check(st, "moe_fp8_matmul")
    M, N = y.shape
    K = x.shape[-1]
    kb = -(-K // FP8_GROUP)
    px, ldx = _rows(x, _F8, "x", M, K)
    pw, ldw = _rows(w, _F8, "w", N, K)
    py, ldy = _rows(y, _BF16, "y", M, N)
    pxs, pws = _dense(x_scales, _F32, "x_scales", M * kb), _dense(w_scales, _F32, "w_scales", -(-N // FP8_GROUP) * kb)
    perr = _dense(err_flag, _I32, "err_flag")
    _check_device(stream, x, x_scales, w, w_scales, y, err_flag)
    _check((_lib or lib()).moe_fp8_matmul(px, ldx, pxs, pw, ldw, pws, py, ldy, M, N, K, perr, _raw_stream(stream, y)),
           "moe_fp8_matmul")


def _grouped_operands(x, x_scales, w, w_scales, y, topk_weights, x_per_pair):
    M, topk, N = y.shape
    E, _, K = w.shape
    kb = -(-K // FP8_GROUP)
    rows = M * topk if x_per_pair else M
    px, ldx = _rows(x, _F8, "x", rows, K)
    pw, ldw = _rows(w, _F8, "w", E * N, K)
    py, ldy = _rows(y, _BF16, "y", M * topk, N)
    return M, topk, E, K, N, (px, 1 if x_per_pair else 0, ldx, _dense(x_scales, _F32, "x_scales", rows * kb), pw, ldw,
                              _dense(w_scales, _F32, "w_scales", E * -(-N // FP8_GROUP) * kb), py, ldy,
                              _dense(topk_weights, _F32, "topk_weights", M * topk))


def fp8_grouped_workspace_bytes(M, topk, num_experts, K, N, block_size) -> int:
    """Bytes of workspace of a moe_fp8_grouped_matmul call with these sizes."""
    return lib().moe_fp8_grouped_workspace_bytes(M, topk, num_experts, K, N, block_size)


def _take_workspace(nbytes, y, stream, raw):
    """nbytes of torch's allocator for a call on `stream` (raw: its handle)."""
    if not nbytes:
        return None
    workspace = torch.empty(nbytes, dtype=torch.uint8, device=y.device)
    if stream is not None:
        # the allocator's earlier work on this memory is ordered on the current stream, its next on either
        side = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(raw, y.device)
        side.wait_stream(torch.cuda.current_stream(y.device))
        workspace.record_stream(side)
    return workspace


def moe_fp8_grouped_matmul(x, x_scales, w, w_scales, y, sorted_token_ids, expert_ids, num_tokens_post_padded,
                           block_size, topk_weights=None, x_per_pair=False, workspace=None, err_flag=None,
                           stream=None):
    """moe_fp8_matmul over a MoE layer's experts, on moe_align_block_size's
    blocks; see include/moe_lora.h.

    x: float8_e4m3fn [M, K] ([M*topk, K] with x_per_pair); w: float8_e4m3fn [E,
    N, K], w_scales: float32 [E, ceil(N / 128), ceil(K / 128)]; y: bf16 [M,
    topk, N], written in place for every pair of a block and no other (zero it
    first where the align drops pairs and all rows are read); topk_weights: float32
    [M, topk] or None.  workspace: a uint8 tensor of at least
    fp8_grouped_workspace_bytes(...) bytes; without one, calls that need one
    take it from torch's allocator."""
    if stream is None and workspace is None:
        st = (_fast or _load_fast()).grouped(x, x_scales, w, w_scales, y, topk_weights, bool(x_per_pair), err_flag,
                                           sorted_token_ids, expert_ids, num_tokens_post_padded, block_size)
        if st is not None:
            return _check(st, "moe_fp8_grouped_matmul")
    M, topk, E, K, N, operands = _grouped_operands(x, x_scales, w, w_scales, y, topk_weights, x_per_pair)
    blocks = [_dense(t, _I32, name) for t, name in (
        (sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
        (num_tokens_post_padded, "num_tokens_post_padded"))]
    perr = _dense(err_flag, _I32, "err_flag")
    _check_device(stream, x, x_scales, w, w_scales, y, topk_weights, sorted_token_ids, expert_ids,
                  num_tokens_post_padded, workspace, err_flag)
    L = _lib or lib()
    raw = _raw_stream(stream, y)
    nbytes = 0
    if workspace is None:
        nbytes = L.moe_fp8_grouped_workspace_bytes(M, topk, E, K, N, block_size)
        workspace = _take_workspace(nbytes, y, stream, raw)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    _check(L.moe_fp8_grouped_matmul(
        *operands, *blocks, M, topk, E, K, N, block_size, sorted_token_ids.numel(), expert_ids.numel(),
        None if workspace is None else _dense(workspace, workspace.dtype, "workspace"), nbytes, perr, raw),
        "moe_fp8_grouped_matmul")


def moe_fp8_grouped_matmul_naive(x, x_scales, w, w_scales, y, topk_ids, topk_weights=None, x_per_pair=False,
                                 err_flag=None, stream=None):
    """moe_fp8_grouped_matmul without an align, one work item per (token,
    top-k) pair; topk_ids: int32 [M, topk]."""
    if stream is None:
        st = (_fast or _load_fast()).naive(x, x_scales, w, w_scales, y, topk_weights, bool(x_per_pair), err_flag, topk_ids)
        if st is not None:
            return _check(st, "moe_fp8_grouped_matmul_naive")
    M, topk, E, K, N, operands = _grouped_operands(x, x_scales, w, w_scales, y, topk_weights, x_per_pair)
    pids, perr = _dense(topk_ids, _I32, "topk_ids", M * topk), _dense(err_flag, _I32, "err_flag")
    _check_device(stream, x, x_scales, w, w_scales, y, topk_weights, topk_ids, err_flag)
    _check((_lib or lib()).moe_fp8_grouped_matmul_naive(*operands, pids, M, topk, E, K, N, perr, _raw_stream(stream, y)),
           "moe_fp8_grouped_matmul_naive")


def _either(t, name, numel):
    """Address of a contiguous bf16 or fp32 CUDA tensor, and whether it is fp32 (None: none)."""
    if t is None:
        return None, 0
    if t.dtype is not _BF16 and t.dtype is not _F32:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))
    return _dense(t, t.dtype, name, numel), int(t.dtype is _F32)


def moe_route(logits, topk_ids, topk_weights, bias=None, scoring=ROUTE_SOFTMAX, renormalize=True, scale=1.0,
              num_groups=1, topk_groups=1, group_best=1, stream=None):
    """Each token's top-k experts and their weights; see include/moe_lora.h.

    logits: bf16 or float32 [M, E], rows may be strided.  topk_ids: int32 [M,
    topk] and topk_weights: float32 [M, topk], written.  bias: float32 [E] or
    None, added to the scores for the choice alone.  scoring: ROUTE_SOFTMAX or
    ROUTE_SIGMOID."""
    if stream is None:
        st = (_fast or _load_fast()).route(logits, topk_ids, topk_weights, bias, scoring, renormalize, scale, num_groups,
                                           topk_groups, group_best)
        if st is not None:
            return _check(st, "moe_route")
    M, E = logits.shape
    topk = topk_ids.shape[-1]
    if logits.dtype is not _BF16 and logits.dtype is not _F32:
        raise TypeError("logits must be bfloat16 or float32, got %s" % logits.dtype)
    pl, ld = _rows(logits, logits.dtype, "logits", M, E)
    pi, pw = _dense(topk_ids, _I32, "topk_ids", M * topk), _dense(topk_weights, _F32, "topk_weights", M * topk)
    pb = _dense(bias, _F32, "bias", E)
    _check_device(stream, logits, topk_ids, topk_weights, bias)
    _check((_lib or lib()).moe_route(pl, int(logits.dtype is _F32), max(ld, E), pb, scoring, int(bool(renormalize)), scale,
                                     num_groups, topk_groups, group_best, pi, pw, M, E, topk,
                                     _raw_stream(stream, topk_ids)), "moe_route")


def moe_bf16_matmul(x, w, y, bias=None, residual=None, activation=ACT_NONE, err_flag=None, stream=None):
    """y = activation(x @ w.T + bias) + residual; see include/moe_lora.h.

    x: bf16 [M, K]; w: bf16 [N, K]; y: bf16 or float32 [M, N]; bias: bf16 or
    float32 [N] or None; residual: of y's type, [M, N], or None (may be y).
    Rows of x, w, residual and y may be strided (x, w: by multiples of 8).
    activation: ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU or ACT_GELU_TANH."""
    if stream is None:
        st = (_fast or _load_fast()).matmul16(x, w, y, bias, residual, activation, err_flag)
        if st is not None:
            return _check(st, "moe_bf16_matmul")
    M, N = y.shape
    K = x.shape[-1]
    if y.dtype is not _BF16 and y.dtype is not _F32:
        raise TypeError("y must be bfloat16 or float32, got %s" % y.dtype)
    px, ldx = _rows(x, _BF16, "x", M, K)
    pw, ldw = _rows(w, _BF16, "w", N, K)
    py, ldy = _rows(y, y.dtype, "y", M, N)
    pr, ldr = (None, 0) if residual is None else _rows(residual, y.dtype, "residual", M, N)
    pb, bias_f32 = _either(bias, "bias", N)
    perr = _dense(err_flag, _I32, "err_flag")
    _check_device(stream, x, w, y, bias, residual, err_flag)
    _check((_lib or lib()).moe_bf16_matmul(px, ldx, pw, ldw, pb, bias_f32, pr, ldr, py, ldy, int(y.dtype is _F32),
                                           activation, M, N, K, perr, _raw_stream(stream, y)), "moe_bf16_matmul")


def _grouped16_operands(x, w, y, bias, activation, topk_weights, x_per_pair):
    M, topk, N = y.shape
    E, _, K = w.shape
    px, ldx = _rows(x, _BF16, "x", M * topk if x_per_pair else M, K)
    pw, ldw = _rows(w, _BF16, "w", E * N, K)
    py, ldy = _rows(y, _BF16, "y", M * topk, N)
    pb, bias_f32 = _either(bias, "bias", E * N)
    return M, topk, E, K, N, (px, 1 if x_per_pair else 0, ldx, pw, ldw, pb, bias_f32, py, ldy, activation,
                              _dense(topk_weights, _F32, "topk_weights", M * topk))


def bf16_grouped_workspace_bytes(M, topk, num_experts, K, N, block_size) -> int:
    """Bytes of workspace of a moe_bf16_grouped_matmul call with these sizes."""
    return lib().moe_bf16_grouped_workspace_bytes(M, topk, num_experts, K, N, block_size)


def moe_bf16_grouped_matmul(x, w, y, sorted_token_ids, expert_ids, num_tokens_post_padded, block_size, bias=None,
                            activation=ACT_NONE, topk_weights=None, x_per_pair=False, workspace=None, err_flag=None,
                            stream=None):
    """activation(x @ w[e].T + bias[e]) over a MoE layer's experts, on
    moe_align_block_size's blocks; see include/moe_lora.h.

    x: bf16 [M, K] ([M*topk, K] with x_per_pair); w: bf16 [E, N, K]; bias: bf16
    or float32 [E, N] or None; y: bf16 [M, topk, N], written in place for every
    pair of a block and no other (zero it first where the align drops pairs and
    all rows are read); topk_weights: float32 [M, topk] or None.  workspace: a
    uint8 tensor of at least bf16_grouped_workspace_bytes(...) bytes; without
    one, calls that need one take it from torch's allocator."""
    if stream is None and workspace is None:
        st = (_fast or _load_fast()).grouped16(x, w, y, bias, activation, topk_weights, bool(x_per_pair), err_flag,
                                               sorted_token_ids, expert_ids, num_tokens_post_padded, block_size)
        if st is not None:
            return _check(st, "moe_bf16_grouped_matmul")
    M, topk, E, K, N, operands = _grouped16_operands(x, w, y, bias, activation, topk_weights, x_per_pair)
    blocks = [_dense(t, _I32, name) for t, name in (
        (sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
        (num_tokens_post_padded, "num_tokens_post_padded"))]
    perr = _dense(err_flag, _I32, "err_flag")
    _check_device(stream, x, w, y, bias, topk_weights, sorted_token_ids, expert_ids, num_tokens_post_padded, workspace,
                  err_flag)
    L = _lib or lib()
    raw = _raw_stream(stream, y)
    if workspace is None:
        nbytes = L.moe_bf16_grouped_workspace_bytes(M, topk, E, K, N, block_size)
        workspace = _take_workspace(nbytes, y, stream, raw)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    _check(L.moe_bf16_grouped_matmul(
        *operands, *blocks, M, topk, E, K, N, block_size, sorted_token_ids.numel(), expert_ids.numel(),
        None if workspace is None else _dense(workspace, workspace.dtype, "workspace"), nbytes, perr, raw),
        "moe_bf16_grouped_matmul")


def moe_bf16_grouped_matmul_naive(x, w, y, topk_ids, bias=None, activation=ACT_NONE, topk_weights=None,
                                  x_per_pair=False, err_flag=None, stream=None):
    """moe_bf16_grouped_matmul without an align, one work item per (token,
    top-k) pair; topk_ids: int32 [M, topk]."""
    if stream is None:
        st = (_fast or _load_fast()).naive16(x, w, y, bias, activation, topk_weights, bool(x_per_pair), err_flag, topk_ids)
        if st is not None:
            return _check(st, "moe_bf16_grouped_matmul_naive")
    M, topk, E, K, N, operands = _grouped16_operands(x, w, y, bias, activation, topk_weights, x_per_pair)
    pids, perr = _dense(topk_ids, _I32, "topk_ids", M * topk), _dense(err_flag, _I32, "err_flag")
    _check_device(stream, x, w, y, bias, topk_weights, topk_ids, err_flag)
    _check((_lib or lib()).moe_bf16_grouped_matmul_naive(*operands, pids, M, topk, E, K, N, perr, _raw_stream(stream, y)),
           "moe_bf16_grouped_matmul_naive")


class AlignBuffers:
    """Device output buffers (and workspace) for one align configuration."""

    def __init__(self, M, topk, num_experts, max_loras, num_active_loras, block_size, device="cuda",
                 variant=ALIGN_AUTO):
        cap = max_num_tokens_padded(M, topk, num_experts, block_size)
        capb = max_num_m_blocks(M, topk, num_experts, block_size)
        self.sorted_token_ids = torch.empty((max_loras, cap), dtype=torch.int32, device=device)
        self.expert_ids = torch.empty((max_loras, capb), dtype=torch.int32, device=device)
        self.num_tokens_post_padded = torch.empty((max_loras,), dtype=torch.int32, device=device)
        nbytes = align_workspace_bytes(M, topk, num_experts, num_active_loras, block_size, variant)
        self.workspace = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=device) if nbytes else None
