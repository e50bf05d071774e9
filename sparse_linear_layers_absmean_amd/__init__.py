"""Sparse-BitLinear (W1.58A8, N:M) for AMD MI355X.

The compute path lives in libsbl.so (HIP kernels for gfx950 behind the C ABI
declared in include/sbl.h); `sbl` is its thin Python binding.  Importing the
package does not load the library: `sbl.load()` (or the first call) does.
"""

from .sbl import (SBL_FMT_DENSE2, SBL_FMT_NM, SblError, linear, load, new_backward_workspace, new_workspace,
                  quant_acts, sbl_backward_workspace_bytes,
                  quant_weights, sbl_abi_version, sbl_linear, sbl_linear_acts_batch, sbl_linear_backward,
                  sbl_linear_batch, sbl_linear_grouped, sbl_linear_kgrouped, sbl_meta_bytes,
                  sbl_linear_blocked, sbl_quant_acts_kgrouped, sbl_quant_weights_blocked,
                  sbl_quant_weights_grouped, sbl_workspace_bytes_blocked, sbl_workspace_bytes_grouped,
                  sbl_pack,
                  sbl_packed_bytes, sbl_quant_acts, sbl_quant_weights, sbl_quant_weights_batch,
                  sbl_quant_weights_batch_noalloc,
                  sbl_workspace_bytes,
                  sbl_workspace_init,
                  SBL_BF16, SBL_FP16, head_ce, head_ce_backward, head_kd, head_kd_backward, new_head_workspace,
                  sbl_head_ce_backward, sbl_head_ce_forward, sbl_head_kd_backward, sbl_head_kd_forward,
                  sbl_head_workspace_bytes,
                  SBL_FP32, AdamWItems, adamw_schedule, adamw_state, embed, embed_backward, join_master,
                  new_embed_workspace, new_norm_workspace, norm, norm_backward, norm_quant, sbl_adamw_batch,
                  sbl_embed_backward, sbl_embed_forward, sbl_embed_workspace_bytes, sbl_norm_backward,
                  sbl_norm_forward, sbl_norm_workspace_bytes, split_master)

__all__ = [
    "SBL_FMT_DENSE2", "SBL_FMT_NM", "SblError", "linear", "load", "new_backward_workspace", "new_workspace",
    "quant_acts", "sbl_backward_workspace_bytes",
    "quant_weights", "sbl_abi_version", "sbl_linear", "sbl_linear_acts_batch", "sbl_linear_backward",
    "sbl_linear_batch", "sbl_linear_grouped", "sbl_linear_kgrouped", "sbl_meta_bytes",
    "sbl_linear_blocked", "sbl_quant_acts_kgrouped", "sbl_quant_weights_blocked",
    "sbl_quant_weights_grouped", "sbl_workspace_bytes_blocked", "sbl_workspace_bytes_grouped",
    "sbl_pack",
    "sbl_packed_bytes", "sbl_quant_acts", "sbl_quant_weights", "sbl_quant_weights_batch",
    "sbl_quant_weights_batch_noalloc",
    "sbl_workspace_bytes",
    "sbl_workspace_init",
    "SBL_BF16", "SBL_FP16", "head_ce", "head_ce_backward", "head_kd", "head_kd_backward", "new_head_workspace",
    "sbl_head_ce_backward", "sbl_head_ce_forward", "sbl_head_kd_backward", "sbl_head_kd_forward",
    "sbl_head_workspace_bytes",
    "SBL_FP32", "AdamWItems", "adamw_schedule", "adamw_state", "embed", "embed_backward", "join_master",
    "new_embed_workspace", "new_norm_workspace", "norm", "norm_backward", "norm_quant", "sbl_adamw_batch",
    "sbl_embed_backward", "sbl_embed_forward", "sbl_embed_workspace_bytes", "sbl_norm_backward",
    "sbl_norm_forward", "sbl_norm_workspace_bytes", "split_master",
]
