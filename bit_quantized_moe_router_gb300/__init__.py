"""GB300 (sm_103a) Q2_K mixture-of-experts FFN layer.

The layer runs in hand-written CUDA kernels behind the C ABI of
include/qs_moe.h (libqs_moe.so); `qs_moe` is its Python binding.
"""
from . import build
from . import qs_moe
from .qs_moe import (QS_BF16, QS_E4M3, QS_F32, Cache, QsError, Seqs, alloc_cache_attention_workspace, alloc_dispatch_workspace, alloc_fp8_matmul_workspace,
                     alloc_rmsnorm_backward_workspace, alloc_workspace, make_cache, make_experts, make_seqs, make_shape,
                     make_shared, qs_cache_attention, qs_cache_read, qs_cache_write,
                     qs_combine_tokens, qs_combine_tokens_backward, qs_dispatch_tokens, qs_fp8_matmul,
                     qs_group_tokens, qs_moe_ffn, qs_moe_workspace_bytes, qs_q2k_down_combine,
                     qs_q2k_gemv_grouped, qs_q2k_quantize, qs_read_device_status, qs_rmsnorm_residual,
                     qs_rmsnorm_residual_backward, qs_route_topk, qs_shared_expert_ffn, qs_silu_mul_quant,
                     qs_workspace_init)

__all__ = ["Cache", "Seqs", "alloc_cache_attention_workspace", "make_cache", "make_seqs", "qs_cache_attention", "qs_cache_read",
           "qs_cache_write", "build", "qs_moe", "QS_BF16", "QS_E4M3", "QS_F32", "QsError", "alloc_dispatch_workspace",
           "alloc_fp8_matmul_workspace", "alloc_rmsnorm_backward_workspace", "qs_combine_tokens",
           "qs_combine_tokens_backward", "qs_dispatch_tokens", "qs_fp8_matmul", "qs_rmsnorm_residual",
           "qs_rmsnorm_residual_backward", "qs_silu_mul_quant", "alloc_workspace", "make_experts", "make_shape",
           "make_shared", "qs_group_tokens", "qs_moe_ffn", "qs_moe_workspace_bytes", "qs_q2k_down_combine",
           "qs_q2k_gemv_grouped", "qs_q2k_quantize", "qs_read_device_status", "qs_route_topk",
           "qs_shared_expert_ffn", "qs_workspace_init"]
