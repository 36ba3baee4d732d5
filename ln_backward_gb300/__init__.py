"""GB300-native memory-bound training-step kernels.

``libtb.so`` (built from ``csrc/`` for sm_103a) implements the fused
mixed-precision multi-tensor AdamW step, the row-wise softmax backward, the
LayerNorm and RMSNorm backward, rotary positions with the per-head norm of
queries and keys, causal attention, the gated projections of a feed-forward
block and the output layer's cross entropy behind the C ABI declared in
``include/tb.h``.  This package is its thin Python binding (same names as the C entry points) plus the seeded
synthetic-input module ``synth``.
"""
from ._binding import (  # noqa: F401
    EXPORTS, STATUS, TB_BF16, TB_F16, TB_F32, AdamWPlan, TbError, library_path,
    tb_adamw_grad_norm, tb_adamw_grad_norm_workspace_size, tb_adamw_plan_create,
    tb_adamw_plan_destroy, tb_adamw_selftest_stale_counter, tb_adamw_step, tb_adamw_step_clipped,
    tb_adamw_step_device,
    tb_attention, tb_attention_bwd, tb_attention_bwd_workspace_size,
    tb_attention_selftest_timeout,
    tb_cast_from_f32, tb_cast_to_f32,
    tb_device_error,
    tb_gated_linear, tb_gated_linear_bwd, tb_gated_linear_bwd_workspace_size,
    tb_gated_linear_selftest_timeout, tb_gated_linear_workspace_size,
    tb_layernorm_bwd, tb_layernorm_bwd_noalloc, tb_layernorm_bwd_selftest_timeout,
    tb_layernorm_bwd_workspace_size,
    tb_linear_xent, tb_linear_xent_bwd, tb_linear_xent_bwd_workspace_size,
    tb_linear_xent_selftest_timeout, tb_linear_xent_workspace_size,
    tb_qk_norm_rope, tb_qk_norm_rope_bwd, tb_qk_norm_rope_bwd_workspace_size,
    tb_rmsnorm_bwd, tb_rmsnorm_bwd_workspace_size,
    tb_rope, tb_rope_bwd, tb_rope_freqs, tb_softmax_bwd, tb_softmax_bwd_causal,
    tb_status_string, tb_version,
)
