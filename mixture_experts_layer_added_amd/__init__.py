"""MI355X (gfx950) DeepSeekMoE layer forward with aux-loss-free load balancing.

The computation runs in libmoe.so (hand-written HIP kernels behind a C ABI declared
in include/moe.h); this package holds the ctypes binding (`_lib`), a buffer-owning
layer object (`layer.MoELayer`) and the build script (`build`).
"""
from ._lib import (MoeError, moe_balance_loss, moe_balance_loss_backward, moe_bias_update,  # noqa: F401
                   moe_checkpoint_restore, moe_checkpoint_save, moe_combine, moe_expert_ffn,
                   moe_expert_ffn_backward_input_checkpoint, moe_gemm_fp8, moe_permute,
                   moe_quantize_fp8, moe_quantize_weights_fp8, moe_route,
                   moe_router_backward_dense, moe_workspace_bytes, problem,
                   moe_collect, moe_collect_backward, moe_dequantize_mxfp4, moe_dispatch,
                   moe_dispatch_backward, moe_expert_ffn_down_mxfp4, moe_expert_ffn_up_mxfp4,
                   moe_gemm_mxfp4, moe_pack_expert_weights_mxfp4, moe_quantize_mxfp4,
                   moe_sort_by_expert)

__all__ = ["MoeError", "moe_route", "moe_permute", "moe_expert_ffn", "moe_combine",
           "moe_bias_update", "moe_quantize_weights_fp8", "moe_workspace_bytes", "problem",
           "moe_balance_loss", "moe_balance_loss_backward", "moe_router_backward_dense",
           "moe_checkpoint_save", "moe_checkpoint_restore",
           "moe_expert_ffn_backward_input_checkpoint", "moe_quantize_fp8", "moe_gemm_fp8",
           "moe_quantize_mxfp4", "moe_dequantize_mxfp4", "moe_gemm_mxfp4",
           "moe_pack_expert_weights_mxfp4", "moe_expert_ffn_up_mxfp4",
           "moe_expert_ffn_down_mxfp4", "moe_sort_by_expert", "moe_dispatch",
           "moe_dispatch_backward", "moe_collect", "moe_collect_backward"]
