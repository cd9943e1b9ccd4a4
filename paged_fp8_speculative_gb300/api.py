"""Python binding of the C ABI (argument marshalling only).

Every function has the name of the C entry point it calls.  PyTorch supplies
device memory and the current stream; every step of the computation runs in
the library's CUDA kernels.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import torch

from ._lib import lib

HEAD_DIM = 256
PAGE_SIZE = 16
MAX_SEGMENTS = 64

OK, E_ARG, E_UNSUPPORTED, E_DEVICE, E_WORKSPACE, E_LAUNCH = 0, -1, -2, -3, -4, -5
E_SCRATCH_LIMIT = -6
STATIC_SCRATCH_BYTES = 32 << 20
ERR_QLEN, ERR_QLEN_GT_SEQ, ERR_PAGE, ERR_SEQ_TOO_LONG, ERR_TIMEOUT = 1, 2, 4, 8, 16
WORKSPACE_HEADER_BYTES = 4352     # MTPATTN_WORKSPACE_HEADER_BYTES: tile and call counters


class MtpAttnError(RuntimeError):
    def __init__(self, code: int):
        self.code = code
        super().__init__(f"mtpattn status {code}: {mtp_verify_attn_strerror(code)}")


def mtp_verify_attn_strerror(code: int) -> str:
    return lib().mtp_verify_attn_strerror(int(code)).decode()


def mtp_verify_attn_num_segments(num_seqs: int, num_kv_heads: int, max_pages_per_seq: int,
                                 device: int = -1) -> int:
    r = lib().mtp_verify_attn_num_segments(num_seqs, num_kv_heads, max_pages_per_seq, device)
    if r < 0:
        raise MtpAttnError(r)
    return r


def mtp_verify_attn_workspace_size(total_q: int, num_q_heads: int, num_segments: int) -> int:
    return int(lib().mtp_verify_attn_workspace_size(total_q, num_q_heads, num_segments))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _temporaries_on(stream, device, needed: bool):
    """Context for the temporaries a wrapper makes for a call (descale tensors from Python
    floats, a zeroed workspace, out, lse): when the call runs on a stream other than the
    current one, they are made on that stream, so that they are written in its order, before
    the library's kernels read them, and their memory is not handed out again while those
    kernels may still use it.  Nothing to do when the call makes none, or runs on the current
    stream (entering a stream context costs microseconds of host time per call)."""
    if not needed or stream is None or device.type != "cuda":
        return contextlib.nullcontext()
    ts = stream if isinstance(stream, torch.cuda.Stream) else \
        torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(ts)


def _descale(x, device) -> torch.Tensor:
    if isinstance(x, torch.Tensor):
        return x
    return torch.full((1,), float(x), dtype=torch.float32, device=device)


def _check_args(q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, kd, vd, out):
    """The shape, dtype and layout checks both entry points share (the C side checks
    pointers, strides, alignment and the envelope, but cannot see shapes)."""
    if q.dtype != torch.bfloat16 or q.dim() != 3 or q.shape[2] != HEAD_DIM or q.stride(2) != 1:
        raise ValueError("q must be bf16 [total_q, H_q, 256] with unit stride on head_dim")
    if k_cache.dtype not in (torch.uint8, torch.float8_e4m3fn) or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache / v_cache must be uint8 or float8_e4m3fn codes")
    if k_cache.dim() != 4 or k_cache.shape[1] != PAGE_SIZE or k_cache.shape[3] != HEAD_DIM:
        raise ValueError("k_cache must be [num_pages, 16, H_kv, 256]")
    if v_cache.shape != k_cache.shape or not k_cache.is_contiguous() or not v_cache.is_contiguous():
        raise ValueError("k_cache and v_cache must be contiguous and of the same shape")
    for name, t in (("block_tables", block_tables), ("seq_lens", seq_lens),
                    ("cu_seqlens_q", cu_seqlens_q)):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor")
    num_seqs = seq_lens.numel()
    if seq_lens.dim() != 1 or block_tables.dim() != 2 or block_tables.shape[0] != num_seqs or \
            cu_seqlens_q.dim() != 1 or cu_seqlens_q.numel() != num_seqs + 1:
        raise ValueError("block_tables [B, max_pages], seq_lens [B], cu_seqlens_q [B+1]")
    for name, t in (("k_descale", kd), ("v_descale", vd)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.numel() != 1:
            raise ValueError(f"{name} must be a 1-element float32 tensor")
    total_q, hq, _ = q.shape
    if out is not None and (out.dtype != torch.bfloat16 or tuple(out.shape) != (total_q, hq, HEAD_DIM)
                            or out.stride(2) != 1):
        raise ValueError("out must be bf16 [total_q, H_q, 256] with unit stride on head_dim")
    return num_seqs, total_q, hq, k_cache.shape[2]


def _verify_fwd(entry, q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, k_descale,
                v_descale, softmax_scale, num_segments, out, workspace, status, stream):
    dev = q.device
    makes = (out is None or workspace is None or not isinstance(k_descale, torch.Tensor) or
             not isinstance(v_descale, torch.Tensor))
    with _temporaries_on(stream, dev, makes):
        kd = _descale(k_descale, dev)
        vd = _descale(v_descale, dev)
        num_seqs, total_q, hq, hkv = _check_args(q, k_cache, v_cache, block_tables, seq_lens,
                                                 cu_seqlens_q, kd, vd, out)
        # None / 0: the library chooses S (and may then share the partial slots out by
        # length); a workspace made here is sized for the S it will choose, a given one is
        # checked by the library.
        chosen = int(num_segments or 0)
        if workspace is not None and not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")     # (taken as the bytes from its first one on)
        if out is None:
            out = torch.empty(total_q, hq, HEAD_DIM, dtype=torch.bfloat16, device=dev)
        if workspace is None:
            S = chosen or mtp_verify_attn_num_segments(num_seqs, hkv, block_tables.shape[1],
                                                       dev.index if dev.index is not None else -1)
            need = mtp_verify_attn_workspace_size(total_q, hq, S)
            workspace = torch.zeros(max(need, 256), dtype=torch.uint8, device=dev)
    rc = entry(
        _ptr(q), q.stride(0), q.stride(1),
        _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
        _ptr(block_tables), block_tables.shape[1],
        _ptr(seq_lens), _ptr(cu_seqlens_q),
        num_seqs, total_q, hq, hkv,
        _ptr(kd), _ptr(vd), float(softmax_scale), chosen,
        _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(out), out.stride(0), out.stride(1),
        _ptr(status), _stream_handle(stream))
    if rc != OK:
        raise MtpAttnError(rc)
    return out


def mtp_verify_attn_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        block_tables: torch.Tensor, seq_lens: torch.Tensor,
                        cu_seqlens_q: torch.Tensor, k_descale, v_descale,
                        softmax_scale: float, num_segments: Optional[int] = None,
                        out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Paged fp8 verify / draft-extend / decode attention; returns ``out`` (bf16).

    q [total_q, H_q, 256] bf16; k_cache / v_cache [num_pages, 16, H_kv, 256]
    uint8 or float8_e4m3fn codes; block_tables [B, max_pages] int32; seq_lens [B]
    int32; cu_seqlens_q [B+1] int32; descales 1-element float32 device tensors
    (a Python float is copied to the device).  ``num_segments`` None or 0 lets the library
    choose S; a long sequence may then take more than S pieces when short ones use fewer
    (the workspace's rows x S partial slots are shared out by length).  ``status`` is an optional int32
    device word that collects device-side error bits (ERR_*).  Without ``workspace`` a zeroed
    one is allocated for this call; a decode loop passes its own (zeroed once, reused by every
    call on the stream) so that no call allocates.
    """
    return _verify_fwd(lib().mtp_verify_attn_fwd, q, k_cache, v_cache, block_tables, seq_lens,
                       cu_seqlens_q, k_descale, v_descale, softmax_scale, num_segments, out,
                       workspace, status, stream)


def mtp_verify_attn_fwd_qp_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               block_tables: torch.Tensor, seq_lens: torch.Tensor,
                               cu_seqlens_q: torch.Tensor, k_descale, v_descale,
                               softmax_scale: float, num_segments: Optional[int] = None,
                               out: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None,
                               status: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """mtp_verify_attn_fwd with Q and P rounded once to e4m3 (the pages' precision class,
    about 0.15 std of error instead of 0.01); planned scheduling only, so batches of more
    (sequence, KV head) units than SMs raise MtpAttnError(E_UNSUPPORTED)."""
    return _verify_fwd(lib().mtp_verify_attn_fwd_qp_fp8, q, k_cache, v_cache, block_tables,
                       seq_lens, cu_seqlens_q, k_descale, v_descale, softmax_scale,
                       num_segments, out, workspace, status, stream)


def mtp_verify_attn_fwd_static_scratch(q: torch.Tensor, k_cache: torch.Tensor,
                                       v_cache: torch.Tensor, block_tables: torch.Tensor,
                                       seq_lens: torch.Tensor, cu_seqlens_q: torch.Tensor,
                                       k_descale: torch.Tensor, v_descale: torch.Tensor,
                                       softmax_scale: float, num_segments: int, out: torch.Tensor,
                                       status: Optional[torch.Tensor] = None,
                                       stream=None) -> torch.Tensor:
    """The attention without a caller workspace, for callers that cannot allocate.

    The split-KV partials go to the library's own static device array
    (STATIC_SCRATCH_BYTES per GPU), so this wrapper allocates nothing either:
    ``out``, the descale tensors (1-element float32 device tensors, not Python
    floats) and every input are the caller's, and they get the same checks as in
    mtp_verify_attn_fwd.  Calls that overlap on the GPU share that array and race;
    serialise them.
    """
    if out is None:
        raise ValueError("out is required: this entry point allocates nothing")
    num_seqs, total_q, hq, hkv = _check_args(q, k_cache, v_cache, block_tables, seq_lens,
                                             cu_seqlens_q, k_descale, v_descale, out)
    rc = lib().mtp_verify_attn_fwd_static_scratch(
        _ptr(q), q.stride(0), q.stride(1),
        _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
        _ptr(block_tables), block_tables.shape[1],
        _ptr(seq_lens), _ptr(cu_seqlens_q),
        num_seqs, total_q, hq, hkv,
        _ptr(k_descale), _ptr(v_descale), float(softmax_scale), int(num_segments),
        _ptr(out), out.stride(0), out.stride(1),
        _ptr(status), _stream_handle(stream))
    if rc != OK:
        raise MtpAttnError(rc)
    return out


def mtp_verify_attn_set_deterministic(on: bool) -> None:
    """Fixed page ranges per piece (bit-identical repeats) instead of balanced tile sharing."""
    lib().mtp_verify_attn_set_deterministic(1 if on else 0)


def mtp_verify_attn_get_deterministic() -> bool:
    return bool(lib().mtp_verify_attn_get_deterministic())


SCHED_CHUNKED = 0
SCHED_PLANNED = 1


def mtp_verify_attn_set_scheduling(mode: int) -> None:
    """Chunked (0, sized for max_pages) or planned (1, sized from seq_lens on the device)."""
    rc = lib().mtp_verify_attn_set_scheduling(int(mode))
    if rc != OK:
        raise ValueError(f"unknown scheduling mode {mode}")


def mtp_verify_attn_get_scheduling() -> int:
    return int(lib().mtp_verify_attn_get_scheduling())


def mtpattn_stream_read(buf: torch.Tensor, sink: Optional[torch.Tensor] = None, blocks: int = 0,
                        stream=None) -> torch.Tensor:
    """Read every byte of ``buf`` once (streaming-read ceiling probe); returns the sink (int32, one word a block)."""
    if not buf.is_contiguous():
        raise ValueError("buf must be contiguous")
    if blocks == 0:
        blocks = int(lib().mtpattn_stream_read_default_blocks())
        if blocks <= 0:
            raise MtpAttnError(blocks)
    with _temporaries_on(stream, buf.device, sink is None):
        if sink is None:
            sink = torch.empty(blocks, dtype=torch.int32, device=buf.device)
    if sink.dtype != torch.int32 or not sink.is_contiguous() or sink.numel() < blocks:
        raise ValueError(f"sink must be a contiguous int32 tensor of at least {blocks} words")
    nbytes = buf.numel() * buf.element_size()
    rc = lib().mtpattn_stream_read(_ptr(buf), nbytes, _ptr(sink), blocks, _stream_handle(stream))
    if rc != OK:
        raise MtpAttnError(rc)
    return sink


# ---- fp8 varlen prefill (include/fmha_fp8_varlen.h) ---------------------------------------------

HEAD_DIM_QK = 192
HEAD_DIM_V = 128
ERR_CU = 32


def fmha_fwd_fp8_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_descale, k_descale,
                        v_descale, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                        max_seqlen_q: int, max_seqlen_k: int, softmax_scale: Optional[float] = None,
                        is_causal: bool = False, return_lse: bool = False,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream=None):
    """fp8 varlen prefill attention (q/k head dim 192, v 128); returns out, or (out, lse).

    q [total_q, H_q, 192], k [total_k, H_kv, 192], v [total_k, H_kv, 128]: uint8 or
    float8_e4m3fn codes with unit stride on the head dim; cu_seqlens_q / cu_seqlens_k int32
    [B+1]; descales 1-element float32 device tensors (a Python float is copied to the
    device); softmax_scale defaults to 1/sqrt(192); out bf16 [total_q, H_q, 128]; lse float32
    [H_q, total_q] (natural log), allocated when return_lse and not given.
    """
    for name, t, d in (("q", q, HEAD_DIM_QK), ("k", k, HEAD_DIM_QK), ("v", v, HEAD_DIM_V)):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or t.dim() != 3 or t.shape[2] != d \
                or t.stride(2) != 1:
            raise ValueError(f"{name} must be e4m3 codes [rows, heads, {d}] with unit stride on "
                             "the head dim")
    if k.shape[:2] != v.shape[:2]:
        raise ValueError("k and v must have the same rows and heads")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if t.dtype != torch.int32 or not t.is_contiguous() or t.dim() != 1:
            raise ValueError(f"{name} must be a contiguous int32 vector")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both have num_seqs + 1 entries")
    dev = q.device
    makes = (out is None or (return_lse and lse is None) or
             not all(isinstance(x, torch.Tensor) for x in (q_descale, k_descale, v_descale)))
    with _temporaries_on(stream, dev, makes):
        qd, kd, vd = (_descale(x, dev) for x in (q_descale, k_descale, v_descale))
        for name, t in (("q_descale", qd), ("k_descale", kd), ("v_descale", vd)):
            if t.dtype != torch.float32 or t.numel() != 1:
                raise ValueError(f"{name} must be a 1-element float32 tensor")
        total_q, hq, _ = q.shape
        total_k, hkv, _ = k.shape
        if out is None:
            out = torch.empty(total_q, hq, HEAD_DIM_V, dtype=torch.bfloat16, device=dev)
        if out.dtype != torch.bfloat16 or tuple(out.shape) != (total_q, hq, HEAD_DIM_V) or \
                out.stride(2) != 1:
            raise ValueError("out must be bf16 [total_q, H_q, 128] with unit stride on the head "
                             "dim")
        if return_lse and lse is None:
            lse = torch.empty(hq, total_q, dtype=torch.float32, device=dev)
        if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (hq, total_q)
                                or not lse.is_contiguous()):
            raise ValueError("lse must be a contiguous float32 [H_q, total_q] tensor")
    scale = 1.0 / math.sqrt(HEAD_DIM_QK) if softmax_scale is None else float(softmax_scale)
    rc = lib().fmha_fwd_fp8_varlen(
        _ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0), k.stride(1),
        _ptr(v), v.stride(0), v.stride(1), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
        cu_seqlens_q.numel() - 1, total_q, total_k, int(max_seqlen_q), int(max_seqlen_k), hq, hkv,
        _ptr(qd), _ptr(kd), _ptr(vd), scale, 1 if is_causal else 0,
        _ptr(out), out.stride(0), out.stride(1), _ptr(lse), _ptr(status), _stream_handle(stream))
    if rc != OK:
        raise MtpAttnError(rc)
    return (out, lse) if return_lse else out


# ---- draft trees (include/mtp_tree.h) ------------------------------------------------------------
#
# These calls are short, so their checks, the outputs that are not given and the call itself are in
# csrc/binding.cpp (arguments by position; None: not given).

TREE_MAX_NODES = 64
TREE_MAX_RATIO = 16
TREE_MAX_VOCAB = 1 << 20
ERR_PARENT, ERR_ROW = 64, 128

_BINDING = None


def binding():
    """The compiled part of the binding (raises RuntimeError if it has not been built)."""
    global _BINDING
    if _BINDING is None:
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError("the compiled binding is missing or does not load "
                               f"({e}): build it with `python -m paged_fp8_speculative_gb300.build`")
        _binding.set_error(MtpAttnError)
        _BINDING = _binding
    return _BINDING


def _on_stream(call, args, stream, device):
    """``call`` on a stream that was given: its handle goes last, and what the call makes is made on
    that stream (see _temporaries_on)."""
    if isinstance(stream, torch.cuda.Stream):
        if device.type == "cuda" and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, tensors are on {device}")
        handle = stream.cuda_stream
    else:
        handle = int(stream)
    with _temporaries_on(stream, device, True):
        return call(*args, handle)


def mtp_tree_mask(parents: torch.Tensor, cu_seqlens_q: torch.Tensor,
                  out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """One word per node of the packed draft trees: its ancestors' bits and its own.

    parents [total_q] int32 (an index within the sequence; the root's entry is not read);
    cu_seqlens_q [B+1] int32; returns int64 [total_q] (the bits of the uint64 words).
    """
    call = (_BINDING or binding()).tree_mask
    if stream is None:
        return call(parents, cu_seqlens_q, out, status, None)
    return _on_stream(call, (parents, cu_seqlens_q, out, status), stream, parents.device)


def mtp_tree_attn_workspace_size(num_seqs: int, total_q: int, num_q_heads: int,
                                 num_kv_heads: int, max_pages_per_seq: int) -> int:
    return int(lib().mtp_tree_attn_workspace_size(num_seqs, total_q, num_q_heads, num_kv_heads,
                                                  max_pages_per_seq))


def mtp_tree_attn_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, seq_lens: torch.Tensor,
                      cu_seqlens_q: torch.Tensor, tree_mask: torch.Tensor, k_descale, v_descale,
                      softmax_scale: float, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of trees of 1 to 64 drafted tokens over the paged fp8 cache; returns ``out``.

    As mtp_verify_attn_fwd, with any GQA ratio from 1 to 16 and ``tree_mask`` [total_q] int64:
    node t sees every key before its sequence's tree (the last cu_seqlens_q[b+1] -
    cu_seqlens_q[b] cached tokens) and the tree's node i where bit i of its word is set
    (mtp_tree_mask makes the words).  A node that sees nothing gets zeros.  ``workspace``: at
    least mtp_tree_attn_workspace_size(...) bytes, kept by a decode loop so that no call
    allocates; it needs no initialisation.
    """
    call = (_BINDING or binding()).tree_attn
    if not (isinstance(k_descale, torch.Tensor) and isinstance(v_descale, torch.Tensor)):
        with _temporaries_on(stream, q.device, True):
            k_descale, v_descale = _descale(k_descale, q.device), _descale(v_descale, q.device)
    if stream is None:
        return call(q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, tree_mask,
                    k_descale, v_descale, softmax_scale, out, workspace, status, None)
    return _on_stream(call, (q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, tree_mask,
                             k_descale, v_descale, softmax_scale, out, workspace, status), stream,
                      q.device)


def mtp_tree_verify_greedy(logits: torch.Tensor, draft_tokens: torch.Tensor,
                           parents: torch.Tensor, cu_seqlens_q: torch.Tensor,
                           max_path: int = TREE_MAX_NODES,
                           accept_index: Optional[torch.Tensor] = None,
                           accept_len: Optional[torch.Tensor] = None,
                           out_tokens: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, stream=None):
    """The path of drafted tokens that are their parents' argmax.

    logits [total_q, vocab] float32, bfloat16 or float16 (the target's, after each node);
    draft_tokens, parents [total_q] int32; returns (accept_index [B, max_path] int32: the
    root's 0, the accepted nodes, -1s; accept_len [B] int32; out_tokens [B, max_path] int32: the
    accepted tokens, the next token, -1s).
    """
    call = (_BINDING or binding()).verify_greedy
    if stream is None:
        return call(logits, draft_tokens, parents, cu_seqlens_q, max_path, accept_index,
                    accept_len, out_tokens, status, None)
    return _on_stream(call, (logits, draft_tokens, parents, cu_seqlens_q, max_path, accept_index,
                             accept_len, out_tokens, status), stream, logits.device)


def mtp_tree_verify_sample(target_probs: torch.Tensor, draft_probs: Optional[torch.Tensor],
                           draft_tokens: torch.Tensor, parents: torch.Tensor,
                           cu_seqlens_q: torch.Tensor, uniforms: torch.Tensor,
                           max_path: int = TREE_MAX_NODES,
                           accept_index: Optional[torch.Tensor] = None,
                           accept_len: Optional[torch.Tensor] = None,
                           out_tokens: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, stream=None):
    """The path by rejection sampling from given uniform numbers.

    target_probs [total_q, vocab] float32, bfloat16 or float16: the target's distribution after
    each node; draft_probs the same shape and type, row i the distribution node i's children
    were drawn from, or None (children chosen outright); uniforms [total_q] float32 in [0, 1):
    each node's own number, the root's for the final draw.  Returns as mtp_tree_verify_greedy.
    """
    call = (_BINDING or binding()).verify_sample
    if stream is None:
        return call(target_probs, draft_probs, draft_tokens, parents, cu_seqlens_q, uniforms,
                    max_path, accept_index, accept_len, out_tokens, status, None)
    return _on_stream(call, (target_probs, draft_probs, draft_tokens, parents, cu_seqlens_q,
                             uniforms, max_path, accept_index, accept_len, out_tokens, status),
                      stream, target_probs.device)


# ---- the paged cache's upkeep (include/mtp_cache.h; checks and calls in csrc/binding.cpp) ---------

CACHE_MAX_ROWS = 8192
ERR_LEN, ERR_FULL, ERR_REF, ERR_CACHE_ROW = 256, 512, 1024, 2048


def mtp_cache_workspace_size(num_rows: int, max_pages_per_seq: int) -> int:
    return int(lib().mtp_cache_workspace_size(num_rows, max_pages_per_seq))


def mtp_cache_resize(k_cache: torch.Tensor, v_cache: Optional[torch.Tensor], block_tables: torch.Tensor,
                     seq_lens: torch.Tensor, ref_counts: torch.Tensor, new_lens: torch.Tensor,
                     workspace: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Set every row's length, in place: pages are given back and handed out.

    k_cache / v_cache: one layer's caches [num_pages, 16, H_kv, 256] or a stack's, behind
    num_layers; or latent vectors [num_pages, 16, 576], or a stack of them, with v_cache None (here
    and in the calls below); block_tables [rows, max_pages], seq_lens [rows], ref_counts [num_pages] int32 are
    updated; new_lens [rows] int32 (0 frees a row).  A shared, partly filled last page is copied
    first.  With too few free pages nothing is handed out and ERR_FULL is set.
    """
    call = (_BINDING or binding()).cache_resize
    if stream is None:
        return call(k_cache, v_cache, block_tables, seq_lens, ref_counts, new_lens, workspace,
                    status, None)
    return _on_stream(call, (k_cache, v_cache, block_tables, seq_lens, ref_counts, new_lens,
                             workspace, status), stream, block_tables.device)


def mtp_cache_fork(k_cache: torch.Tensor, v_cache: Optional[torch.Tensor], block_tables: torch.Tensor,
                   seq_lens: torch.Tensor, ref_counts: torch.Tensor, src: torch.Tensor,
                   dst: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Rows dst[i] (empty) become copies of rows src[i]: full pages are shared, a partly filled
    last page is copied.  src, dst int32 vectors of the same length."""
    call = (_BINDING or binding()).cache_fork
    if stream is None:
        return call(k_cache, v_cache, block_tables, seq_lens, ref_counts, src, dst, workspace,
                    status, None)
    return _on_stream(call, (k_cache, v_cache, block_tables, seq_lens, ref_counts, src, dst,
                             workspace, status), stream, block_tables.device)


def mtp_cache_copy_pages(k_cache: torch.Tensor, v_cache: Optional[torch.Tensor], src_pages: torch.Tensor,
                         dst_pages: torch.Tensor, status: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """Page dst_pages[i] gets the contents of page src_pages[i], in all layers."""
    call = (_BINDING or binding()).cache_copy_pages
    if stream is None:
        return call(k_cache, v_cache, src_pages, dst_pages, status, None)
    return _on_stream(call, (k_cache, v_cache, src_pages, dst_pages, status), stream,
                      k_cache.device)


def mtp_cache_compact(k_cache: torch.Tensor, v_cache: Optional[torch.Tensor], block_tables: torch.Tensor,
                      seq_lens: torch.Tensor, cu_seqlens_q: torch.Tensor,
                      accept_index: torch.Tensor, accept_len: torch.Tensor,
                      new_seq_lens: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Move the accepted paths' keys and values to the front of their trees' places, in all
    layers, in place; returns new_seq_lens [B] int32 (the tokens kept).

    accept_index [B, max_path] and accept_len [B] as the verifications return them.  The pages
    that hold the trees must belong to their rows alone; none are given back here.
    """
    call = (_BINDING or binding()).cache_compact
    if stream is None:
        return call(k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, accept_index,
                    accept_len, new_seq_lens, status, None)
    return _on_stream(call, (k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, accept_index,
                             accept_len, new_seq_lens, status), stream, k_cache.device)


# ---- rotary positions and new tokens (include/mtp_rope.h; checks and calls in csrc/binding.cpp) ------


def mtp_rope_freqs(inv_freq, device=None) -> torch.Tensor:
    """The angles of rotary positions as the calls below take them: int64 [pairs], whole numbers of
    2^-64 turns a position, from radians a position (``inv_freq``: numbers or a tensor, 0 to 2^20;
    rope.inv_freq makes the usual ones).  Made once and kept."""
    values = inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else [float(x) for x in inv_freq]
    n = len(values)
    radians, out = (ctypes.c_double * n)(*values), (ctypes.c_int64 * n)()
    rc = lib().mtp_rope_freqs(ctypes.cast(radians, ctypes.c_void_p), n, ctypes.cast(out, ctypes.c_void_p))
    if rc != OK:
        raise ValueError("inv_freq must be finite, 0 to 2^20 radians a position")
    return torch.tensor(list(out), dtype=torch.int64, device=device)


def _descales(device, stream, *values):
    with _temporaries_on(stream, device, True):
        return tuple(_descale(x, device) for x in values)


def mtp_rope_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                    positions: torch.Tensor, freqs: Optional[torch.Tensor], k_cache: torch.Tensor,
                    v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                    cu_seqlens_q: torch.Tensor, k_descale, v_descale, mscale: float = 1.0,
                    interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """New tokens into one layer's K/V cache, with rotary positions on q and k; returns q_out.

    q [total_q, H_q, 256] (None: no q), k and v [total_q, H_kv, 256]: bfloat16, float16 or float32, all
    the same, unit stride along the head (views of a joint projection will do); positions [total_q]
    int32; freqs int64 [pairs] (mtp_rope_freqs; the first 2 * pairs elements of a head are rotated, a
    multiple of 16; None: none); the caches, tables, lengths (the new tokens included) and cu_seqlens_q
    of the attention calls, with any number of tokens a sequence; descales as there.  Pairs are elements
    2i and 2i + 1 (interleaved) or i and i + pairs; mscale is a factor on sines and cosines.  q_out
    (bf16) may be q itself.
    """
    call = (_BINDING or binding()).rope_append
    if not (isinstance(k_descale, torch.Tensor) and isinstance(v_descale, torch.Tensor)):
        k_descale, v_descale = _descales(k.device, stream, k_descale, v_descale)
    if stream is None:
        return call(q, k, v, positions, freqs, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q,
                    k_descale, v_descale, mscale, interleaved, q_out, status, None)
    return _on_stream(call, (q, k, v, positions, freqs, k_cache, v_cache, block_tables, seq_lens,
                             cu_seqlens_q, k_descale, v_descale, mscale, interleaved, q_out, status),
                      stream, k.device)


def mtp_rope_latent_append(q_rope: Optional[torch.Tensor], latent: torch.Tensor,
                           k_rope: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor,
                           cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                           cu_seqlens_q: torch.Tensor, descale, mscale: float = 1.0,
                           interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None,
                           stream=None) -> Optional[torch.Tensor]:
    """New tokens into a latent cache (mtp_latent_attn_fwd reads it); returns q_out.

    latent [total_q, 512] and k_rope [total_q, 64] (rotated on the way) become the 576 codes of a token
    in cache [num_pages, 16, 576]; q_rope [total_q, H, 64] (None: no q) is rotated into q_out (bf16;
    pass the last 64 elements of the attention's rows of 576, or q_rope itself).  All else as in
    mtp_rope_append; freqs has 32 entries.
    """
    call = (_BINDING or binding()).rope_latent_append
    if not isinstance(descale, torch.Tensor):
        descale, = _descales(latent.device, stream, descale)
    if stream is None:
        return call(q_rope, latent, k_rope, positions, freqs, cache, block_tables, seq_lens,
                    cu_seqlens_q, descale, mscale, interleaved, q_out, status, None)
    return _on_stream(call, (q_rope, latent, k_rope, positions, freqs, cache, block_tables, seq_lens,
                             cu_seqlens_q, descale, mscale, interleaved, q_out, status), stream,
                      latent.device)


def mtp_rope_prefill(q: torch.Tensor, k: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor,
                     positions: torch.Tensor, freqs: torch.Tensor, q_descale, k_descale, v_descale,
                     mscale: float = 1.0, interleaved: bool = False,
                     q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                     v_out: Optional[torch.Tensor] = None, stream=None):
    """fmha_fwd_fp8_varlen's operands from the projections' outputs; returns (q, k, v) as e4m3 codes.

    q [tokens, H_q, 192] (its last 64 elements are rotated), k [tokens, H_kv, 128], k_rope [tokens, 64]
    (rotated, shared by all heads), v [tokens, H_kv, 128]: bfloat16, float16 or float32, all the same;
    freqs has 32 entries.  The outputs are contiguous [tokens, H_q, 192], [tokens, H_kv, 192] and
    [tokens, H_kv, 128].
    """
    call = (_BINDING or binding()).rope_prefill
    if not (isinstance(q_descale, torch.Tensor) and isinstance(k_descale, torch.Tensor) and
            isinstance(v_descale, torch.Tensor)):
        q_descale, k_descale, v_descale = _descales(q.device, stream, q_descale, k_descale, v_descale)
    if stream is None:
        return call(q, k, k_rope, v, positions, freqs, q_descale, k_descale, v_descale, mscale,
                    interleaved, q_out, k_out, v_out, None)
    return _on_stream(call, (q, k, k_rope, v, positions, freqs, q_descale, k_descale, v_descale, mscale,
                             interleaved, q_out, k_out, v_out), stream, q.device)


# ---- latent attention (include/mtp_latent.h) ------------------------------------------------------

LATENT_DIM, LATENT_ROPE_DIM, LATENT_MAX_HEADS = 512, 64, 128


def mtp_latent_attn_workspace_size(num_seqs: int, total_q: int, num_heads: int,
                                   max_pages_per_seq: int) -> int:
    return int(lib().mtp_latent_attn_workspace_size(num_seqs, total_q, num_heads, max_pages_per_seq))


def mtp_latent_attn_fwd(q: torch.Tensor, cache: torch.Tensor, block_tables: torch.Tensor,
                        seq_lens: torch.Tensor, cu_seqlens_q: torch.Tensor, descale,
                        softmax_scale: float, tree_mask: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of 1 to 64 new tokens a sequence over a paged cache of latent vectors, in the absorbed
    form; returns ``out`` [total_q, H, 512] bf16.

    q [total_q, H, 576] bf16, H to 128: a head's query in the latent space, then its rotated part (64);
    cache [num_pages, 16, 576] uint8 or float8_e4m3fn codes, with ``descale``; tables, lengths and
    cu_seqlens_q as in mtp_verify_attn_fwd.  Token i of a sequence's new ones (its last in the cache)
    sees what is before them and the new ones up to itself, or those of its word of ``tree_mask``
    [total_q] int64 (mtp_tree_mask).  ``workspace``: at least mtp_latent_attn_workspace_size(...) bytes,
    kept by a decode loop so that no call allocates (made for the largest batch, it does for all); it needs
    no initialisation.
    """
    call = (_BINDING or binding()).latent_attn
    if not isinstance(descale, torch.Tensor):
        descale, = _descales(q.device, stream, descale)
    if stream is None:
        return call(q, cache, block_tables, seq_lens, cu_seqlens_q, descale, softmax_scale, tree_mask, out,
                    workspace, status, None)
    return _on_stream(call, (q, cache, block_tables, seq_lens, cu_seqlens_q, descale, softmax_scale,
                             tree_mask, out, workspace, status), stream, q.device)
