"""GB300-native attention over packed, ragged THD batches: forward, backward
and the sparse-attention indexer top-k; the per-head norm with the position rotation
that feeds it; page tables and one-token attention over a paged cache.

The compute path is the C-ABI library ``libthd_attn.so`` (CUDA kernels for
sm_103a); :mod:`.binding`, :mod:`.norm_rope` and :mod:`.paged` marshal torch
tensors into its calls. Importing this package does not load the library; the
first call does, and fails loudly when the library has not been built.
"""
from .binding import (STATS_HEAD_MAJOR, STATS_TOKEN_MAJOR, KERNEL_AUTO, KERNEL_SIMT,
                      KERNEL_MMA, KERNEL_TCGEN05, ThdAttnError, ThdAttnPlan, alloc_workspace, library_path,
                      load_library,
                      ThdAttention, thd_attention, thd_attn_backward, thd_attn_forward, thd_attn_fwd,
                      thd_attn_plan, thd_attn_read_status, thd_indexer)
from .norm_rope import (FLAG_ZERO_SKIPPED, ThdQkNormRope, qk_norm_rope_bwd_plan_for_tensors,
                        qk_norm_rope_paged_plan_for_tensors, qk_norm_rope_plan_for_tensors, thd_qk_norm_rope,
                        thd_qk_norm_rope_append, thd_qk_norm_rope_backward, thd_qk_norm_rope_bwd,
                        thd_qk_norm_rope_forward, thd_qk_norm_rope_fwd, thd_qk_norm_rope_paged)
from .paged import (paged_decode_plan_for_tensors, paged_tables_plan, thd_paged_attention, thd_paged_decode,
                    thd_paged_extend, thd_paged_tables)

__all__ = [
    "STATS_HEAD_MAJOR", "STATS_TOKEN_MAJOR", "KERNEL_AUTO", "KERNEL_SIMT", "KERNEL_TCGEN05",
    "ThdAttnError", "ThdAttnPlan", "library_path", "load_library", "thd_attn_forward",
    "thd_attn_fwd", "thd_attn_plan", "thd_attn_read_status", "thd_attn_backward", "thd_indexer",
    "ThdAttention", "thd_attention", "KERNEL_MMA", "alloc_workspace",
    "FLAG_ZERO_SKIPPED", "ThdQkNormRope", "qk_norm_rope_bwd_plan_for_tensors", "qk_norm_rope_paged_plan_for_tensors",
    "qk_norm_rope_plan_for_tensors", "thd_qk_norm_rope", "thd_qk_norm_rope_append", "thd_qk_norm_rope_backward",
    "thd_qk_norm_rope_bwd", "thd_qk_norm_rope_forward", "thd_qk_norm_rope_fwd", "thd_qk_norm_rope_paged",
    "paged_decode_plan_for_tensors", "paged_tables_plan", "thd_paged_attention", "thd_paged_decode",
    "thd_paged_extend", "thd_paged_tables",
]
