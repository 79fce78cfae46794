"""GB300 (sm_103a) fused attention forward: a C-ABI CUDA library and its
Python binding.

``forward`` computes O = softmax(scale * Q K^T + causal mask) V and the per-row
log-sum-exp with one persistent tcgen05/TMA kernel (and, with split-KV, a
small merge kernel); ``prepare`` fixes the tensors and options of a call so
that repeated calls skip the argument marshalling. ``cache_append``,
``cache_read`` and ``paged_forward`` keep the keys and values of sequences that
grow in a paged cache (bf16, e4m3 or 4 bits) and attend to it; ``rotary`` turns
queries and keys by their positions (``cache_append`` does so on the way), with
the angles of ``rotary_table``. Build the library with
``attention_forward_sm100_gb300.build.build()``.
"""
from ._binding import (AttnError, Params, PlanInfo, PreparedForward, check, default_workspace, forward, key_range,
                       last_error, lib, make_params, paged_native, plan, prepare, schedule, workspace_bytes)
from .paged import cache_append, cache_read, paged_forward
from .rope import rotary, rotary_frequencies, rotary_table

__all__ = ["AttnError", "Params", "PlanInfo", "PreparedForward", "cache_append", "cache_read", "check",
           "default_workspace", "forward", "key_range", "last_error", "lib", "make_params", "paged_forward",
           "paged_native", "plan", "prepare", "rotary", "rotary_frequencies", "rotary_table", "schedule",
           "workspace_bytes"]
