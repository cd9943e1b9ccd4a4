"""Paged fp8 split-KV attention for speculative-decoding verify, draft extend and
decode on GB300 (sm_103a), the attention and verification of draft trees, and the
paged cache's upkeep: a C-ABI CUDA library (libmtpattn.so) and its thin
Python binding.  The entry points load the library on first use and
raise if it has not been built."""
from .api import (MtpAttnError, mtp_cache_compact, mtp_cache_copy_pages, mtp_cache_fork,
                  mtp_cache_resize, mtp_cache_workspace_size, mtp_tree_attn_fwd,
                  mtp_tree_attn_workspace_size, mtp_tree_mask, mtp_tree_verify_greedy,
                  mtp_tree_verify_sample, mtp_verify_attn_fwd, mtp_verify_attn_num_segments,
                  mtp_verify_attn_strerror, mtp_verify_attn_workspace_size, mtpattn_stream_read)

__all__ = ["MtpAttnError", "mtp_cache_compact", "mtp_cache_copy_pages", "mtp_cache_fork",
           "mtp_cache_resize", "mtp_cache_workspace_size", "mtp_tree_attn_fwd",
           "mtp_tree_attn_workspace_size", "mtp_tree_mask", "mtp_tree_verify_greedy",
           "mtp_tree_verify_sample", "mtp_verify_attn_fwd", "mtp_verify_attn_num_segments",
           "mtp_verify_attn_strerror", "mtp_verify_attn_workspace_size", "mtpattn_stream_read"]
