"""MI355X (gfx950) sparse Mixture-of-Experts layer forward.

The layer runs in hand-written HIP kernels behind the C ABI of
``include/moe.h``; this package holds those sources (``csrc/``), the build
script and a thin ctypes binding whose functions carry the C names.
"""
from .binding import (DECODE_MAX_TOKENS, DTYPE, MoeError, PATH, SCORE, balance_workspace,  # noqa: F401
                      block_matmul_workspace, channel_matmul_workspace, config_from, load, make_config, make_groups,
                      make_weights, moe_balance, moe_balance_workspace_bytes, moe_block_matmul,
                      moe_block_matmul_workspace_bytes, moe_channel_matmul, moe_channel_matmul_workspace_bytes,
                      moe_combine, moe_config, moe_expert_ffn, moe_groups, moe_layer_forward, moe_layer_forward_grouped,
                      moe_layer_forward_noalloc, moe_permute, moe_prefetch_experts, moe_quantize_rows,
                      moe_quantize_tokens, moe_route, moe_route_backward, moe_route_grouped, moe_select,
                      moe_select_grouped, moe_status_str, moe_topk_rows, moe_workspace_bytes, scale_ld, workspace)
