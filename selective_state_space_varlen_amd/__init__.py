"""Packed variable-length sequence operators of linear-time blocks (Mamba-1's
conv and selective scan, the gated delta rule with its head norms, linear
attention with a decay, layer norm and dropout) on MI355X (gfx950).

The operators are HIP kernels in libssmpack.so behind a C ABI
(include/ssmpack.h); this package is the thin Python binding over it plus a
pipeline helper that chains the calls of one Mamba block's sequence-wise part.
"""
from .binding import (  # noqa: F401
    EXPORTED,
    SSMP_NORM_L2,
    SSMP_NORM_RMS,
    PackPlan,
    SsmpError,
    conv1d_pack_bwd,
    conv1d_pack_bwd_states_workspace_bytes,
    conv1d_pack_bwd_workspace_bytes,
    conv1d_pack_fwd,
    decay_attn_pack_bwd,
    decay_attn_pack_bwd_scratch_bytes,
    decay_attn_pack_fwd,
    decay_attn_pack_fwd_scratch_bytes,
    decay_attn_pack_step,
    dropout_pack_bwd,
    dropout_pack_fwd,
    gated_delta_pack_bwd,
    gated_delta_pack_bwd_scratch_bytes,
    gated_delta_pack_fwd,
    gated_delta_pack_fwd_scratch_bytes,
    gated_delta_pack_saved_bytes,
    gated_delta_pack_step,
    layer_norm_pack_bwd,
    layer_norm_pack_bwd_workspace_bytes,
    layer_norm_pack_fwd,
    load,
    qk_norm_pack_bwd,
    qk_norm_pack_bwd_workspace_bytes,
    qk_norm_pack_fwd,
    selective_scan_pack_bwd,
    selective_scan_pack_bwd_ck,
    selective_scan_pack_bwd_scratch_bytes,
    selective_scan_pack_fwd,
    selective_scan_pack_fwd_ck,
    selective_scan_pack_fwd_noalloc,
    selective_scan_pack_fwd_scratch_bytes,
    selective_scan_pack_saved_bytes,
    selective_scan_pack_workspace_bytes,
    varlen_pack_indices,
    varlen_pack_plan,
)
from .pipeline import backward, decay_backward, decay_forward, delta_backward, delta_forward, forward  # noqa: F401
