/*
 * mtp_tree.h — C ABI of the draft-tree operators in libmtpattn.so (GB300, sm_103a), next to
 * the verify attention of mtpattn.h: the attention of a tree of drafted tokens over the same
 * paged e4m3 cache, and the verification of the drafted tokens against the target model.
 *
 * A draft tree.  Sequence b of a batch has n_b = cu_seqlens_q[b+1] - cu_seqlens_q[b] nodes,
 * 1 <= n_b <= MTP_TREE_MAX_NODES, packed at rows cu_seqlens_q[b] .. of every per-node array.
 * Node 0 is the root: the last token that is known to be right.  Node i > 0 is a drafted
 * token whose parent is node parents[i] (an index within the sequence, 0 <= parents[i] < i;
 * the root's entry is not read).  A chain is the tree parents[i] = i - 1.  The n_b nodes are
 * the last n_b of the sequence's seq_lens[b] cached tokens, in node order.
 *
 * Conventions are those of mtpattn.h: device pointers of the current device, no allocation, no
 * synchronisation, nothing read back on the host (a call may be captured in a CUDA graph),
 * status codes MTPATTN_*, nothing launched on an error return, device-side MTPATTN_ERR_* and
 * MTP_TREE_ERR_* bits OR-ed into the optional status word.  The sources of this library name
 * only the chain of up to four tokens; trees are an extension of its own.
 */
#ifndef MTP_TREE_H
#define MTP_TREE_H

#include <stddef.h>
#include <stdint.h>

#include "mtpattn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MTP_TREE_MAX_NODES 64
#define MTP_TREE_MAX_RATIO 16
#define MTP_TREE_MAX_VOCAB (1 << 20)

/* Element types of logits and probabilities. */
#define MTP_F32 0
#define MTP_BF16 1
#define MTP_F16 2

/* Device-side error bits next to MTPATTN_ERR_QLEN, _QLEN_GT_SEQ, _PAGE, _SEQ_TOO_LONG and
 * _TIMEOUT (mtpattn.h). */
#define MTP_TREE_ERR_PARENT 64   /* parents[i] outside [0, i) */
#define MTP_TREE_ERR_ROW 128     /* a row with nothing to choose from: logits all NaN, or
                                    probabilities without a positive entry */

/*
 * mask[i] = the nodes that node i sees: its ancestors, the root among them, and itself, one bit
 * per node of its sequence.
 *  parents      device int32 [total_q]
 *  cu_seqlens_q device int32 [num_seqs + 1]
 *  mask         device uint64 [total_q], 8-byte aligned
 * A sequence whose node count is outside [1, 64], or whose rows are not within total_q, sets
 * MTPATTN_ERR_QLEN and is not written; a node whose path runs over a bad parent sets
 * MTP_TREE_ERR_PARENT and sees itself and the part of its path below that parent.
 */
int mtp_tree_mask(const int32_t* parents, const int32_t* cu_seqlens_q, int32_t num_seqs,
                  int32_t total_q, uint64_t* mask, int32_t* status, void* stream);

/*
 * Attention of the draft trees over the paged cache:
 *   out[t, h] = v_descale * sum_j softmax_j(softmax_scale * k_descale * <q[t, h], K_j>) V_j
 * over the keys j that node t sees: every key before the tree (j < seq_lens[b] - n_b), and node
 * i of its own sequence where bit i of tree_mask[t] is set (bits >= n_b are ignored; the
 * node's own bit is not implied).  A node that sees no key gets zeros.  Keys that a node does
 * not see do not influence it, whatever codes they hold.
 *
 *  q, k_cache, v_cache, num_pages, block_tables, max_pages_per_seq, seq_lens, k_descale,
 *  v_descale, softmax_scale, out and their strides: as in mtp_verify_attn_fwd (head_dim 256,
 *  page 16, NHD e4m3 pages).  num_q_heads = ratio * num_kv_heads with any ratio in [1, 16].
 *  cu_seqlens_q device int32 [num_seqs + 1], 1 .. 64 nodes each.
 *  tree_mask    device uint64 [total_q], 8-byte aligned.
 *  workspace    device, >= mtp_tree_attn_workspace_size() bytes, 256-byte aligned; need not be
 *               initialised and holds nothing between calls.  Calls that overlap on the GPU
 *               must use different workspaces.
 * Sequences with a device-side error (MTPATTN_ERR_QLEN: node count outside [1, 64];
 * _QLEN_GT_SEQ; _SEQ_TOO_LONG; _PAGE) get zeros, except that the rows of a sequence whose
 * cu_seqlens_q entries are not ascending within total_q are unknown and not written.  (Where the
 * sequences claim more than twice total_q rows in all, nothing is written, with _QLEN.)  Rows
 * that belong to no sequence are not written.  Results are the same bits in every call with the
 * same arguments.  One or two kernels are launched on `stream`.
 */
int mtp_tree_attn_fwd(const void* q, int64_t q_stride_tok, int64_t q_stride_head,
                      const void* k_cache, const void* v_cache, int64_t num_pages,
                      const int32_t* block_tables, int32_t max_pages_per_seq,
                      const int32_t* seq_lens, const int32_t* cu_seqlens_q,
                      const uint64_t* tree_mask, int32_t num_seqs, int32_t total_q,
                      int32_t num_q_heads, int32_t num_kv_heads, const float* k_descale,
                      const float* v_descale, float softmax_scale, void* workspace,
                      size_t workspace_bytes, void* out, int64_t out_stride_tok,
                      int64_t out_stride_head, int32_t* status, void* stream);

/* Bytes of workspace mtp_tree_attn_fwd needs on the current device (0 for invalid arguments or
 * without a device). */
size_t mtp_tree_attn_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_q_heads,
                                    int32_t num_kv_heads, int32_t max_pages_per_seq);

/*
 * Verification, common to both entry points below.  For each sequence a walk starts at the
 * root and follows accepted children; it ends at a node none of whose children is accepted, or
 * after max_path - 1 accepted nodes.
 *  draft_tokens device int32 [total_q] (the root's entry is not read); a token outside
 *               [0, vocab) is never accepted.
 *  max_path     in [1, 64], the width of the outputs.
 *  accept_index device int32 [num_seqs][max_path]: 0 (the root), then the accepted nodes of
 *               the path in order, then -1.
 *  accept_len   device int32 [num_seqs]: the number of accepted drafted tokens.
 *  out_tokens   device int32 [num_seqs][max_path]: the accepted tokens, then the next token
 *               (from the target's row of the last node), then -1.
 * A sequence with a device-side error (MTPATTN_ERR_QLEN, MTP_TREE_ERR_PARENT) gets accept_len
 * -1 and rows of -1.  One kernel is launched.
 */

/*
 * Greedy: a child is accepted if its token is the argmax of its parent's row of logits (ties:
 * the lowest token; of several children with that token the first); the next token is the last
 * node's argmax.  NaN logits are passed over; a row of NaN only sets MTP_TREE_ERR_ROW, and the
 * next token is -1.
 *  logits  device [total_q][vocab] of `dtype` (MTP_F32, _BF16, _F16), row stride `row_stride`
 *          elements (>= vocab), unit stride along the vocabulary, aligned to its element.
 * Only the rows of the nodes on the path are read.
 */
int mtp_tree_verify_greedy(const void* logits, int32_t dtype, int64_t row_stride, int32_t vocab,
                           const int32_t* draft_tokens, const int32_t* parents,
                           const int32_t* cu_seqlens_q, int32_t num_seqs, int32_t total_q,
                           int32_t max_path, int32_t* accept_index, int32_t* accept_len,
                           int32_t* out_tokens, int32_t* status, void* stream);

/*
 * Sampling: rejection sampling from given random numbers.  At a node with the target's row p
 * and the drafter's row q, the children are tried in index order with w = p, Z = 1, S = 0:
 *   child i with token x is accepted if uniforms[i] * q(x) * Z < w(x); if not,
 *   S += Z, w = max(p - S q, 0), Z = sum w.
 * (w / Z is the residual distribution after each refusal.)  Without draft_probs q is 1 at the
 * child's own token and 0 elsewhere: a refused token leaves the row, and Z falls by what it had
 * there.  A token outside [0, vocab) is never accepted.  If no child is accepted the
 * next token is the first x whose running sum of w exceeds uniforms[root] * sum w; if w has no
 * mass left, w = p is used instead, and if p has none, the token is -1 with MTP_TREE_ERR_ROW.
 *  target_probs device [total_q][vocab] of `dtype` (MTP_F32, _BF16 or _F16): row i is the
 *               target's distribution after node i.  Entries are taken into [0, 1]; NaN counts
 *               as 0.
 *  draft_probs  the same layout with its own row stride, or NULL: row i is the distribution
 *               that node i's children were drawn from.
 *  uniforms     device float32 [total_q] in [0, 1): node i's own number, the root's for the
 *               final draw.  Taken into [0, 1 - 2^-24]; NaN counts as 0.
 * Sums are exact: each w is taken to a whole number of units of 2^-45 and these are summed in
 * 64-bit integers, so the result does not depend on the order of summation.  Rows need not sum to
 * 1; a row's sum has to stay below 2^18.
 */
int mtp_tree_verify_sample(const void* target_probs, int64_t target_stride,
                           const void* draft_probs, int64_t draft_stride, int32_t dtype,
                           int32_t vocab, const int32_t* draft_tokens, const int32_t* parents,
                           const int32_t* cu_seqlens_q, const float* uniforms, int32_t num_seqs,
                           int32_t total_q, int32_t max_path, int32_t* accept_index,
                           int32_t* accept_len, int32_t* out_tokens, int32_t* status,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MTP_TREE_H */
