"""GB300-native MoE expert-grouped token reorder.

Two operations behind a C ABI (include/moe_reorder.h), run as hand-written
CUDA kernels for sm_103a:

* ffnwb_batching -- FFN-worker batching: stable counting sort of the slots by
  expert key, row gather (+ INT8 dynamic scale), id lookups, group_list and
  actual_token_num (flat arrays, or a ScheduleContext read on the device);
* moe_permute    -- routing-map permute, the producer of the unpermute's input;
* moe_update_expert -- logical to physical expert ids through the EPLB table,
  with threshold pruning;
* moe_unpermute  -- routing-map unpermute, four branches (padded or not, with
  or without probs), deterministic fp32 gather-reduce;
* moe_quantize, moe_grouped_matmul, moe_expert_ffn -- 8-bit rows and weights
  with a scale per 128 values, the product of each group's rows with its
  expert's weights, and the experts' network between batching and unpermute;
* moe_layer      -- a whole mixture-of-experts layer for up to 64 tokens
  (router, experts, weighted sum) in one launch.

Importing the package does not load the CUDA library; the first call does,
and fails loudly if the library was not built.
"""
from .api import (DT_BF16, DT_E4M3, DT_F16, DT_F32, DT_INT8, MoeReorderError, batching_context_workspace_size,
                  batching_outputs, batching_workspace_size, expert_ffn_workspace_size, ffnwb_batching,
                  ffnwb_batching_context, grouped_matmul_workspace_size, layer_workspace_size, moe_expert_ffn,
                  moe_grouped_matmul, moe_layer, moe_permute, moe_quantize, moe_unpermute, moe_update_expert,
                  permute_workspace_size, profile_set_events, quantize_outputs, unpermute_outputs,
                  unpermute_workspace_size, waits_out)

__all__ = ["ffnwb_batching", "ffnwb_batching_context", "moe_unpermute", "moe_permute", "moe_update_expert",
           "moe_quantize", "moe_grouped_matmul", "moe_expert_ffn", "moe_layer", "quantize_outputs",
           "grouped_matmul_workspace_size", "expert_ffn_workspace_size", "layer_workspace_size", "permute_workspace_size",
           "batching_context_workspace_size", "batching_workspace_size",
           "unpermute_workspace_size", "batching_outputs", "unpermute_outputs",
           "profile_set_events", "waits_out", "MoeReorderError", "DT_F16", "DT_BF16", "DT_INT8", "DT_F32", "DT_E4M3"]
