"""MI355X-native gated delta rule: chunked prefill and its backward pass,
fused recurrent decode (one token or several), the gate computation, and the
short convolution and RMS norms around it; the gated linear recurrence; states and
activations held in 8 or 4 bits.

The compute path is the C-ABI library ``libgdn.so`` (hand-written HIP kernels
for gfx950, declared in ``include/gdn.h``); this package only marshals
arguments to it.
"""
from ._binding import (GDN_BF16, GDN_ERR_SCRATCH, GDN_F32, GDN_OK, GDN_STATIC_SCRATCH_BYTES, LIB_PATH, GdnError, chunk_gated_delta_rule,
                       chunk_gated_delta_rule_bwd, gdn_chunk_bwd, gdn_chunk_bwd_workspace_bytes,
                       fused_gdn_gating, fused_gdn_gating_bwd, fused_recurrent_gated_delta_rule_update, gdn_chunk_fwd,
                       gdn_chunk_fwd_noalloc,
                       gdn_chunk_fwd_gated, gdn_chunk_fwd_pool, gdn_chunk_fwd_workspace_bytes, gdn_decode_shape,
                       gdn_gates, gdn_gating, gdn_gating_bwd, gdn_gating_bwd_workspace_bytes,
                       gdn_profile_enable, gdn_profile_read, gdn_recurrent_update,
                       gdn_recurrent_update_gated, gdn_recurrent_update_pool, gdn_shape, gdn_state_pool,
                       gdn_status_str, load_library, make_decode_shape, make_gates, make_shape, make_state_pool)
from ._binding import EXPORTED as _EXPORTED
from ._binding_layer import (EXPORTED_LAYER, causal_conv1d, causal_conv1d_bwd, causal_conv1d_update,
                             fused_add_rms_norm, fused_add_rms_norm_bwd, fused_gated_rms_norm,
                             fused_gated_rms_norm_bwd, fused_recurrent_gated_delta_rule_steps, gdn_add_norm,
                             gdn_add_norm_bwd, gdn_conv_bwd, gdn_conv_bwd_workspace_bytes, gdn_conv_fwd,
                             gdn_conv_fwd_pool, gdn_conv_pieces, gdn_conv_shape, gdn_conv_update, gdn_gated_norm,
                             gdn_gated_norm_bwd, gdn_norm_bwd_workspace_bytes, gdn_norm_shape, gdn_recurrent_steps,
                             gdn_step_pool, make_step_pool)
from ._binding_scan import (EXPORTED_SCAN, Checkpoint, checkpoint_activation, fused_gated_rms_norm_checkpoint,
                            fused_gated_rms_norm_checkpoint_bwd, gated_linear_recurrence, gated_linear_recurrence_bwd,
                            gated_linear_recurrence_steps, gdn_gated_norm_hold, gdn_gated_norm_hold_bwd, gdn_held,
                            gdn_held_shape, gdn_hold, gdn_restore, gdn_scan_bwd, gdn_scan_fwd, gdn_scan_fwd_pool,
                            gdn_scan_shape, gdn_scan_steps, gdn_scan_workspace_bytes, make_state_cache,
                            restore_activation, state_cache_read, state_cache_write)

EXPORTED = _EXPORTED + EXPORTED_LAYER + EXPORTED_SCAN    # every function of include/gdn.h

__all__ = ["EXPORTED", "GDN_BF16", "GDN_ERR_SCRATCH", "GDN_F32", "GDN_OK", "GDN_STATIC_SCRATCH_BYTES", "LIB_PATH", "GdnError", "chunk_gated_delta_rule",
           "chunk_gated_delta_rule_bwd", "gdn_chunk_bwd", "gdn_chunk_bwd_workspace_bytes",
           "fused_gdn_gating", "fused_gdn_gating_bwd", "fused_recurrent_gated_delta_rule_update", "gdn_chunk_fwd", "gdn_chunk_fwd_noalloc", "gdn_chunk_fwd_gated",
           "gdn_chunk_fwd_pool", "gdn_chunk_fwd_workspace_bytes", "gdn_decode_shape", "gdn_gates", "gdn_gating",
           "gdn_gating_bwd", "gdn_gating_bwd_workspace_bytes",
           "gdn_profile_enable", "gdn_profile_read", "gdn_recurrent_update", "gdn_recurrent_update_gated",
           "gdn_recurrent_update_pool", "gdn_shape", "gdn_state_pool", "gdn_status_str", "load_library",
           "make_decode_shape", "make_gates", "make_shape", "make_state_pool",
           "causal_conv1d", "causal_conv1d_bwd", "causal_conv1d_update", "fused_add_rms_norm",
           "fused_add_rms_norm_bwd", "fused_gated_rms_norm", "fused_gated_rms_norm_bwd",
           "fused_recurrent_gated_delta_rule_steps", "gdn_add_norm", "gdn_add_norm_bwd", "gdn_conv_bwd",
           "gdn_conv_bwd_workspace_bytes", "gdn_conv_fwd", "gdn_conv_fwd_pool", "gdn_conv_pieces", "gdn_conv_shape",
           "gdn_conv_update", "gdn_gated_norm", "gdn_gated_norm_bwd", "gdn_norm_bwd_workspace_bytes",
           "gdn_norm_shape", "gdn_recurrent_steps", "gdn_step_pool", "make_step_pool",
           "Checkpoint", "checkpoint_activation", "fused_gated_rms_norm_checkpoint",
           "fused_gated_rms_norm_checkpoint_bwd", "gated_linear_recurrence", "gated_linear_recurrence_bwd",
           "gated_linear_recurrence_steps", "gdn_gated_norm_hold", "gdn_gated_norm_hold_bwd", "gdn_held",
           "gdn_held_shape", "gdn_hold", "gdn_restore", "gdn_scan_bwd", "gdn_scan_fwd", "gdn_scan_fwd_pool",
           "gdn_scan_shape", "gdn_scan_steps", "gdn_scan_workspace_bytes", "make_state_cache", "restore_activation",
           "state_cache_read", "state_cache_write"]
