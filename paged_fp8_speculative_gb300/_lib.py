"""ctypes loader for libmtpattn.so (the C ABI declared in include/mtpattn.h and
include/fmha_fp8_varlen.h, include/mtp_tree.h, include/mtp_cache.h, include/mtp_rope.h and
include/mtp_latent.h).

There is no fallback: if the library is missing the import of this module's
``lib()`` raises, so no caller can silently run anything else.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmtpattn.so")

_c_int, _c_i32, _c_i64, _c_size, _c_float = (ctypes.c_int, ctypes.c_int32, ctypes.c_int64,
                                             ctypes.c_size_t, ctypes.c_float)
_vp = ctypes.c_void_p

# name -> (restype, argtypes), in the order of include/mtpattn.h, then the other headers
SIGNATURES = {
    "mtp_verify_attn_num_segments": (_c_i32, [_c_i32, _c_i32, _c_i32, _c_i32]),
    "mtp_verify_attn_workspace_size": (_c_size, [_c_i32, _c_i32, _c_i32]),
    "mtp_verify_attn_fwd": (_c_int, [
        _vp, _c_i64, _c_i64,            # q, strides
        _vp, _vp, _c_i64,               # k_cache, v_cache, num_pages
        _vp, _c_i32,                    # block_tables, max_pages_per_seq
        _vp, _vp,                       # seq_lens, cu_seqlens_q
        _c_i32, _c_i32, _c_i32, _c_i32,  # num_seqs, total_q, num_q_heads, num_kv_heads
        _vp, _vp, _c_float, _c_i32,     # k_descale, v_descale, softmax_scale, num_segments
        _vp, _c_size,                   # workspace, workspace_bytes
        _vp, _c_i64, _c_i64,            # out, strides
        _vp, _vp]),                     # status, stream
    "mtp_verify_attn_fwd_qp_fp8": (_c_int, [
        _vp, _c_i64, _c_i64, _vp, _vp, _c_i64, _vp, _c_i32, _vp, _vp,
        _c_i32, _c_i32, _c_i32, _c_i32, _vp, _vp, _c_float, _c_i32,
        _vp, _c_size, _vp, _c_i64, _c_i64, _vp, _vp]),
    "mtp_verify_attn_fwd_static_scratch": (_c_int, [
        _vp, _c_i64, _c_i64, _vp, _vp, _c_i64, _vp, _c_i32, _vp, _vp,
        _c_i32, _c_i32, _c_i32, _c_i32, _vp, _vp, _c_float, _c_i32,
        _vp, _c_i64, _c_i64, _vp, _vp]),
    "mtp_verify_attn_set_deterministic": (None, [_c_i32]),
    "mtp_verify_attn_get_deterministic": (_c_i32, []),
    "mtp_verify_attn_set_scheduling": (_c_i32, [_c_i32]),
    "mtp_verify_attn_get_scheduling": (_c_i32, []),
    "mtp_verify_attn_strerror": (ctypes.c_char_p, [_c_int]),
    "mtpattn_stream_read": (_c_int, [_vp, _c_size, _vp, _c_i32, _vp]),
    "mtpattn_stream_read_default_blocks": (_c_i32, []),
    # include/fmha_fp8_varlen.h
    "fmha_fwd_fp8_varlen": (_c_int, [
        _vp, _c_i64, _c_i64,            # q, strides (bytes)
        _vp, _c_i64, _c_i64,            # k, strides
        _vp, _c_i64, _c_i64,            # v, strides
        _vp, _vp,                       # cu_seqlens_q, cu_seqlens_k
        _c_i32, _c_i32, _c_i32,         # num_seqs, total_q, total_k
        _c_i32, _c_i32,                 # max_seqlen_q, max_seqlen_k
        _c_i32, _c_i32,                 # num_q_heads, num_kv_heads
        _vp, _vp, _vp,                  # q/k/v descales
        _c_float, _c_i32,               # softmax_scale, causal
        _vp, _c_i64, _c_i64,            # out, strides (elements)
        _vp, _vp, _vp]),                # lse, status, stream
    # include/mtp_tree.h
    "mtp_tree_mask": (_c_int, [_vp, _vp, _c_i32, _c_i32, _vp, _vp, _vp]),
    "mtp_tree_attn_fwd": (_c_int, [
        _vp, _c_i64, _c_i64,            # q, strides
        _vp, _vp, _c_i64,               # k_cache, v_cache, num_pages
        _vp, _c_i32,                    # block_tables, max_pages_per_seq
        _vp, _vp, _vp,                  # seq_lens, cu_seqlens_q, tree_mask
        _c_i32, _c_i32, _c_i32, _c_i32,  # num_seqs, total_q, num_q_heads, num_kv_heads
        _vp, _vp, _c_float,             # k_descale, v_descale, softmax_scale
        _vp, _c_size,                   # workspace, workspace_bytes
        _vp, _c_i64, _c_i64,            # out, strides
        _vp, _vp]),                     # status, stream
    "mtp_tree_attn_workspace_size": (_c_size, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32]),
    "mtp_tree_verify_greedy": (_c_int, [
        _vp, _c_i32, _c_i64, _c_i32,    # logits, dtype, row_stride, vocab
        _vp, _vp, _vp,                  # draft_tokens, parents, cu_seqlens_q
        _c_i32, _c_i32, _c_i32,         # num_seqs, total_q, max_path
        _vp, _vp, _vp,                  # accept_index, accept_len, out_tokens
        _vp, _vp]),                     # status, stream
    "mtp_tree_verify_sample": (_c_int, [
        _vp, _c_i64, _vp, _c_i64,       # target_probs, stride, draft_probs, stride
        _c_i32, _c_i32,                 # dtype, vocab
        _vp, _vp, _vp, _vp,             # draft_tokens, parents, cu_seqlens_q, uniforms
        _c_i32, _c_i32, _c_i32,         # num_seqs, total_q, max_path
        _vp, _vp, _vp,                  # accept_index, accept_len, out_tokens
        _vp, _vp]),                     # status, stream
    # include/mtp_cache.h
    "mtp_cache_workspace_size": (_c_size, [_c_i32, _c_i32]),
    "mtp_cache_resize": (_c_int, [
        _vp, _vp, _c_i32, _c_i64, _c_i64, _c_i32,  # caches, layers, layer_stride, pages, kv heads
        _vp, _c_i32, _vp, _c_i32, _vp,  # block_tables, max_pages, seq_lens, num_rows, ref_counts
        _vp, _vp, _c_size,              # new_lens, workspace, workspace_bytes
        _vp, _vp]),                     # status, stream
    "mtp_cache_fork": (_c_int, [
        _vp, _vp, _c_i32, _c_i64, _c_i64, _c_i32,
        _vp, _c_i32, _vp, _c_i32, _vp,
        _vp, _vp, _c_i32, _vp, _c_size,  # src, dst, num_pairs, workspace, workspace_bytes
        _vp, _vp]),
    "mtp_cache_copy_pages": (_c_int, [
        _vp, _vp, _c_i32, _c_i64, _c_i64, _c_i32,
        _vp, _vp, _c_i32,               # src_pages, dst_pages, num_pairs
        _vp, _vp]),
    "mtp_cache_compact": (_c_int, [
        _vp, _vp, _c_i32, _c_i64, _c_i64, _c_i32,
        _vp, _c_i32, _vp, _vp,          # block_tables, max_pages, seq_lens, cu_seqlens_q
        _c_i32, _c_i32,                 # num_seqs, total_q
        _vp, _vp, _c_i32, _vp,          # accept_index, accept_len, max_path, new_seq_lens
        _vp, _vp]),
    # include/mtp_rope.h
    "mtp_rope_freqs": (_c_int, [_vp, _c_i32, _vp]),
    "mtp_rope_append": (_c_int, [
        _vp, _c_i64, _c_i64, _vp, _c_i64, _c_i64, _vp, _c_i64, _c_i64,  # q, k, v, strides
        _c_i32, _vp, _vp,               # dtype, positions, freqs
        _c_i32, _c_i32, _c_float,       # rot_dim, interleaved, mscale
        _vp, _vp, _c_i64, _vp, _c_i32,  # k_cache, v_cache, num_pages, block_tables, max_pages
        _vp, _vp,                       # seq_lens, cu_seqlens_q
        _c_i32, _c_i32, _c_i32, _c_i32,  # num_seqs, total_q, num_q_heads, num_kv_heads
        _vp, _vp,                       # k_descale, v_descale
        _vp, _c_i64, _c_i64,            # q_out, strides
        _vp, _vp]),                     # status, stream
    "mtp_rope_latent_append": (_c_int, [
        _vp, _c_i64, _c_i64,            # q_rope, strides
        _vp, _c_i64, _vp, _c_i64,       # latent, k_rope, strides
        _c_i32, _vp, _vp,               # dtype, positions, freqs
        _c_i32, _c_float,               # interleaved, mscale
        _vp, _c_i64, _vp, _c_i32,       # cache, num_pages, block_tables, max_pages
        _vp, _vp,                       # seq_lens, cu_seqlens_q
        _c_i32, _c_i32, _c_i32,         # num_seqs, total_q, num_heads
        _vp,                            # descale
        _vp, _c_i64, _c_i64,            # q_out, strides
        _vp, _vp]),                     # status, stream
    "mtp_rope_prefill": (_c_int, [
        _vp, _c_i64, _c_i64, _vp, _c_i64, _c_i64,   # q, k, strides
        _vp, _c_i64, _vp, _c_i64, _c_i64,           # k_rope, v, strides
        _c_i32, _vp, _vp, _c_i32, _c_float,         # dtype, positions, freqs, interleaved, mscale
        _c_i32, _c_i32, _c_i32,         # total, num_q_heads, num_kv_heads
        _vp, _vp, _vp,                  # descales
        _vp, _vp, _vp, _vp]),           # q8, k8, v8, stream
    # include/mtp_latent.h
    "mtp_latent_attn_fwd": (_c_int, [
        _vp, _c_i64, _c_i64,            # q, strides
        _vp, _c_i64, _vp, _c_i32,       # cache, num_pages, block_tables, max_pages_per_seq
        _vp, _vp, _vp,                  # seq_lens, cu_seqlens_q, tree_mask
        _c_i32, _c_i32, _c_i32,         # num_seqs, total_q, num_heads
        _vp, _c_float,                  # descale, softmax_scale
        _vp, _c_size,                   # workspace, workspace_bytes
        _vp, _c_i64, _c_i64,            # out, strides
        _vp, _vp]),                     # status, stream
    "mtp_latent_attn_workspace_size": (_c_size, [_c_i32, _c_i32, _c_i32, _c_i32]),
}

_LIB = None


def load(path: str) -> ctypes.CDLL:
    """Load a build of the library at ``path`` with the C signatures attached."""
    handle = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


def lib() -> ctypes.CDLL:
    """The loaded library (raises RuntimeError if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m paged_fp8_speculative_gb300.build`")
        _LIB = load(LIB_PATH)
    return _LIB
