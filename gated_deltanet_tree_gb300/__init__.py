"""State-resident verification of speculative draft trees through Gated DeltaNet layers on GB300, and what a hybrid
model's step needs beside it: attention over a paged 4-bit cache, the acceptance of drafted tokens, prompts and single
tokens through the same layers, and the log-probabilities that the next tree is drafted from.

The computation lives in libgdn_tree.so (hand-written CUDA for sm_103a behind a
C ABI, include/gdn_tree.h).  This package is its ctypes binding plus buffer
ownership; it has no CPU fallback.
"""
from . import _native
from ._native import (GdnError, gdn_abi_version, gdn_accept_workspace_bytes, gdn_attn_dims, gdn_banks, gdn_banks_init,
                      gdn_batch_schedule, gdn_check_error, gdn_check_error_words, gdn_commit_fold, gdn_dims, gdn_finish,
                      gdn_hld_schedule, gdn_kv4_append, gdn_kv4_attention, gdn_kv4_cache, gdn_kv4_pool_bytes,
                      gdn_kv4_read, gdn_kv4_workspace_bytes, gdn_last_error, gdn_pack_schedules, gdn_prefill,
                      gdn_prefill_workspace_bytes, gdn_schedule_words, gdn_step, gdn_top_logprobs, gdn_tree_accept, gdn_tree_verify, gdn_workspace_bytes)
from .build import LIB_PATH

__all__ = ["GdnError", "gdn_abi_version", "gdn_accept_workspace_bytes", "gdn_attn_dims", "gdn_banks", "gdn_banks_init",
           "gdn_batch_schedule", "gdn_check_error", "gdn_check_error_words", "gdn_commit_fold", "gdn_dims", "gdn_finish",
           "gdn_hld_schedule", "gdn_kv4_append", "gdn_kv4_attention", "gdn_kv4_cache", "gdn_kv4_pool_bytes",
           "gdn_kv4_read", "gdn_kv4_workspace_bytes", "gdn_last_error", "gdn_pack_schedules", "gdn_prefill",
           "gdn_prefill_workspace_bytes", "gdn_schedule_words", "gdn_step", "gdn_top_logprobs", "gdn_tree_accept", "gdn_tree_verify", "gdn_workspace_bytes", "LIB_PATH"]
