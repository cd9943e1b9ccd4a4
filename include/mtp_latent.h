/*
 * mtp_latent.h — C ABI of the latent attention in libmtpattn.so (GB300, sm_103a): the decode and verify
 * step of attention whose keys and values are one latent vector a token (the absorbed form; the prefill of
 * fmha_fp8_varlen.h, with its heads of 128 + 64 and 128, is the expanded one).
 *
 * The cache is e4m3 [num_pages][16][576]: a token's latent vector C (512 codes), then its rotated key part
 * R (64 codes), as mtp_rope_latent_append of mtp_rope.h writes them, found through block tables like
 * those of mtpattn.h.  All heads share it.  A query row of 576 is the head's query in the latent space
 * (512: the query times the keys' up-projection) and its rotated part (64).
 *
 * Conventions are those of mtpattn.h: device pointers of the current device, no allocation, no
 * synchronisation, nothing read back (graph-capture safe), status codes MTPATTN_*, nothing launched on an
 * error return, device-side bits OR-ed into the optional status word.
 */
#ifndef MTP_LATENT_H
#define MTP_LATENT_H

#include <stddef.h>
#include <stdint.h>

#include "mtpattn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MTP_LATENT_DIM 512        /* the latent vector: values, and the first elements of a key */
#define MTP_LATENT_ROPE_DIM 64    /* the rotated part of a key */
#define MTP_LATENT_ROW 576
#define MTP_LATENT_MAX_HEADS 128
#define MTP_LATENT_MAX_NODES 64

/*
 *   out[t, h] = descale * sum_j softmax_j(softmax_scale * descale * <q[t, h], (C_j, R_j)>) C_j
 * Sequence b's n_b = cu_seqlens_q[b+1] - cu_seqlens_q[b] new tokens, 1 .. 64, are the last n_b of its
 * seq_lens[b] cached tokens.  New token i sees all tokens before the new ones, and of the new ones those
 * up to itself (tree_mask NULL: a chain), or those whose bit is set in tree_mask (as in mtp_tree_attn_fwd:
 * bits >= n_b are ignored, the token's own bit is not implied).  A token that sees nothing gets zeros.
 * Tokens that a row does not see do not influence it, whatever codes they hold.  Logits are float32: a row of
 * q that holds an infinity or a NaN gets NaN, and so does one that sees a logit (times log2 e) outside float32's range,
 * at either end.
 *
 *  q            device bf16 [total_q][num_heads][576], strides in elements (multiples of 8), unit stride
 *               along the row, 16-byte aligned
 *  cache        device e4m3 [num_pages][16][576], contiguous, 16-byte aligned
 *  block_tables, max_pages_per_seq, seq_lens, cu_seqlens_q   as in mtp_verify_attn_fwd
 *  tree_mask    device uint64 [total_q], 8-byte aligned, or NULL
 *  num_heads    1 .. 128
 *  descale      device float32, one element: of all codes
 *  workspace    device, >= mtp_latent_attn_workspace_size() bytes, 256-byte aligned; need not be
 *               initialised and holds nothing between calls.  Calls that overlap on the GPU must use
 *               different workspaces.
 *  out          device bf16 [total_q][num_heads][512], strides in elements (multiples of 8), 16-byte
 *               aligned; its rows apart from one another and from all inputs
 * Sequences with a device-side error (MTPATTN_ERR_QLEN: n_b outside [1, 64]; _QLEN_GT_SEQ;
 * _SEQ_TOO_LONG; _PAGE) get zeros, except that the rows of a sequence whose cu_seqlens_q entries do not
 * ascend within total_q are unknown and not written.  Rows that belong to no sequence are not written, and rows
 * that several sequences claim (then some entries do not ascend: _QLEN) are unspecified.
 * (MTPATTN_ERR_TIMEOUT: a wait ran out, about two seconds without progress; the rows it concerns are
 * unspecified.)  Results are the same bits in every call with the same arguments.  Two kernels are
 * launched, or one where tables have no more than 32 pages.
 */
int mtp_latent_attn_fwd(const void* q, int64_t q_stride_tok, int64_t q_stride_head, const void* cache,
                        int64_t num_pages, const int32_t* block_tables, int32_t max_pages_per_seq,
                        const int32_t* seq_lens, const int32_t* cu_seqlens_q,
                        const uint64_t* tree_mask, int32_t num_seqs, int32_t total_q,
                        int32_t num_heads, const float* descale, float softmax_scale,
                        void* workspace, size_t workspace_bytes, void* out, int64_t out_stride_tok,
                        int64_t out_stride_head, int32_t* status, void* stream);

/* Bytes of workspace mtp_latent_attn_fwd needs on the current device (0 for invalid arguments or without
 * a device).  It grows with the arguments: a workspace for the largest batch does for all smaller ones. */
size_t mtp_latent_attn_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_heads,
                                      int32_t max_pages_per_seq);

#ifdef __cplusplus
}
#endif

#endif /* MTP_LATENT_H */
