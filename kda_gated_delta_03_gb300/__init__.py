"""Kimi Delta Attention (KDA) operator for one GB300 GPU (sm_103a).

The operator runs in hand-written CUDA kernels behind the C ABI of libkda
(``include/kda.h``); this package is its thin Python binding plus the seeded
input generator (``inputs``) and the build step (``build``).
"""

from .binding import (KdaError, kda_attention_decode, kda_attention_decode_workspace_size, kda_beam_select,
                      kda_beam_select_workspace_size, kda_cache_compact, kda_cache_compact_workspace_size,
                      kda_cache_fork, kda_cache_fork_workspace_size, kda_copy_pages, kda_decode_step,
                      kda_get_device_error, kda_prefill, kda_prefill_backward, kda_prefill_host,
                      kda_prefill_launch_count, kda_prefill_noalloc, kda_prefill_workspace_size, kda_state_fork,
                      kda_status_string, load)

__all__ = ["KdaError", "kda_attention_decode", "kda_attention_decode_workspace_size", "kda_beam_select",
           "kda_beam_select_workspace_size", "kda_cache_compact", "kda_cache_compact_workspace_size", "kda_cache_fork",
           "kda_cache_fork_workspace_size", "kda_copy_pages", "kda_decode_step", "kda_get_device_error", "kda_prefill",
           "kda_prefill_backward", "kda_prefill_host", "kda_prefill_launch_count", "kda_prefill_noalloc",
           "kda_prefill_workspace_size", "kda_state_fork", "kda_status_string", "load"]
