"""GB300-native (sm_103a) exact attention: fused prefill forward and paged-KV decode, with the
norms, rotation, appends and 4-bit cache around it.

The computation lives in the CUDA library ``libattn.so`` (C ABI, include/attn.h);
this package is its thin Python binding.  Importing the package does not load
the library; the first call does, and raises if it has not been built.
"""
from ._binding import (AttnError, LIBRARY_PATH, Q4_BLOCK_BYTES, append_paged, append_paged_q4, debug_inject, decode_paged,
                       decode_paged_append, decode_paged_noalloc, decode_paged_q4, decode_q4_workspace_bytes,
                       decode_workspace_bytes, device_status, fwd, fwd_host, fwd_host_workspace_bytes, fwd_paged,
                       fwd_paged_q4, fwd_paged_q4_workspace_bytes, fwd_simple, fwd_varlen, fwd_workspace_bytes,
                       gather_paged_q4, load, lse_merge, qk_norm_rope, rope_table, selftest_umma, set_wait_budget_ns,
                       set_workspace, status_string, version)

__all__ = ["AttnError", "LIBRARY_PATH", "Q4_BLOCK_BYTES", "append_paged", "append_paged_q4", "debug_inject",
           "decode_paged", "decode_paged_append", "decode_paged_noalloc", "decode_paged_q4",
           "decode_q4_workspace_bytes", "decode_workspace_bytes", "device_status", "fwd", "fwd_host",
           "fwd_host_workspace_bytes", "fwd_paged", "fwd_paged_q4", "fwd_paged_q4_workspace_bytes", "fwd_simple",
           "fwd_varlen", "fwd_workspace_bytes", "gather_paged_q4", "load", "lse_merge", "qk_norm_rope", "rope_table",
           "selftest_umma", "set_wait_budget_ns", "set_workspace", "status_string", "version"]
