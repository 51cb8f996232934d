"""Gated delta rule and selective scan kernels for GB300 (sm_103a): chunked prefill, one-token decode, norms, gradients.

The compute lives in libgdn.so (hand-written CUDA, C ABI in include/gdn.h); this package only
builds it and binds it.  Import is cheap: the library is loaded on the first call.
"""
from ._binding import (  # noqa: F401
    GDN_BF16,
    GDN_F32,
    GDN_FORM_AUTO,
    GDN_FORM_OFF,
    GDN_FORM_ON,
    GDN_NORM_L2,
    GDN_NORM_RMS,
    GdnError,
    gdn_chunk_bwd,
    gdn_chunk_fwd,
    gdn_chunk_fwd_noalloc,
    gdn_decay_from_logits,
    gdn_decay_from_logits_bwd,
    gdn_gate_groupnorm_silu,
    gdn_gate_groupnorm_silu_bwd,
    gdn_gate_rmsnorm_silu,
    gdn_gate_rmsnorm_silu_bwd,
    gdn_get_device_error,
    gdn_qk_norm_rope,
    gdn_qk_norm_rope_bwd,
    gdn_recurrent_multi_step,
    gdn_recurrent_step,
    gdn_selftest_bounded_wait,
    gdn_set_kernel_forms,
    gdn_short_conv_bwd,
    gdn_short_conv_fwd,
    gdn_short_conv_step,
    gdn_ssm_chunk_bwd,
    gdn_ssm_chunk_fwd,
    gdn_ssm_step,
    lib,
)

__all__ = ["gdn_chunk_fwd", "gdn_chunk_fwd_noalloc", "gdn_recurrent_step", "gdn_recurrent_multi_step",
           "gdn_gate_rmsnorm_silu", "gdn_decay_from_logits", "gdn_chunk_bwd", "gdn_gate_rmsnorm_silu_bwd",
           "gdn_gate_groupnorm_silu", "gdn_gate_groupnorm_silu_bwd", "gdn_decay_from_logits_bwd",
           "gdn_short_conv_fwd", "gdn_short_conv_step", "gdn_short_conv_bwd", "gdn_ssm_chunk_fwd", "gdn_ssm_step",
           "gdn_ssm_chunk_bwd", "gdn_qk_norm_rope", "gdn_qk_norm_rope_bwd", "GDN_NORM_RMS", "GDN_NORM_L2",
           "gdn_get_device_error",
           "gdn_selftest_bounded_wait", "gdn_set_kernel_forms", "GdnError", "lib", "GDN_F32", "GDN_BF16",
           "GDN_FORM_AUTO", "GDN_FORM_OFF", "GDN_FORM_ON"]
