"""GB300 (sm_103a) fused attention forward: a C-ABI CUDA library and its
Python binding.

``forward`` computes O = softmax(scale * Q K^T + causal mask) V and the per-row
log-sum-exp with one persistent tcgen05/TMA kernel (and, with split-KV, a
small merge kernel); ``prepare`` fixes the tensors and options of a call so
that repeated calls skip the argument marshalling. ``cache_append``,
``cache_read`` and ``paged_forward`` keep the keys and values of sequences that
grow in a paged cache and attend to it. Build the library with
``attention_forward_sm100_gb300.build.build()``.
"""
from ._binding import (AttnError, Params, PlanInfo, PreparedForward, check, default_workspace, forward, key_range,
                       last_error, lib, make_params, paged_native, plan, prepare, schedule, workspace_bytes)
from .paged import cache_append, cache_read, paged_forward

__all__ = ["AttnError", "Params", "PlanInfo", "PreparedForward", "cache_append", "cache_read", "check",
           "default_workspace", "forward", "key_range", "last_error", "lib", "make_params", "paged_forward",
           "paged_native", "plan", "prepare", "schedule", "workspace_bytes"]
