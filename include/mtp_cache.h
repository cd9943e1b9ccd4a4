/*
 * mtp_cache.h — C ABI of the paged cache's upkeep in libmtpattn.so (GB300, sm_103a): handing
 * out, sharing, copying and giving back the pages that mtp_verify_attn_fwd and
 * mtp_tree_attn_fwd read, and moving the accepted tokens of a draft tree to their places.
 *
 * The cache.  k_cache and v_cache are e4m3 [num_layers][num_pages][16][num_kv_heads][256],
 * contiguous within a layer, layers layer_stride bytes apart (one layer: any stride).  All
 * layers share one block table [num_rows][max_pages_per_seq] (int32, logical page -> physical
 * page; entries at and past ceil(seq_lens / 16) mean nothing and are kept at -1 by these calls),
 * seq_lens [num_rows], and ref_counts [num_pages] (int32): in how many table rows each page
 * stands.  A page with count 0 is free; there is no other list.  A row's last page, if it is
 * only partly filled, belongs to that row alone, so that tokens can be appended in place; full
 * pages may be shared.  mtp_cache_fork and mtp_cache_resize keep that so.
 *
 * Pages are handed out lowest number first, in row order (pair order in a fork) and, within a
 * row, in table order, so equal calls give equal tables.
 *
 * Conventions are those of mtpattn.h: device pointers of the current device, no allocation, no
 * synchronisation, nothing read back (graph-capture safe), nothing launched on an error return,
 * device-side bits OR-ed into the optional status word.  Calls that change the same tables,
 * counts or caches must be ordered by the caller (one stream).
 */
#ifndef MTP_CACHE_H
#define MTP_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "mtpattn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MTP_CACHE_MAX_ROWS 8192
#define MTP_CACHE_MAX_PAGES (1 << 22)   /* of one layer: 8 layers of one head that long fill the GPU */

/* Device-side error bits (next to MTPATTN_ERR_* of mtpattn.h). */
#define MTP_CACHE_ERR_LEN 256    /* a length outside [0, 16 * max_pages_per_seq], or an accepted
                                    path that is not one: the row is left as it was */
#define MTP_CACHE_ERR_FULL 512   /* not enough free pages: nothing was handed out */
#define MTP_CACHE_ERR_REF 1024   /* a page given back had no count left: the count stays 0 */
#define MTP_CACHE_ERR_ROW 2048   /* fork: a row number outside the table, src = dst, a dst that
                                    holds tokens or is named twice: the pair is skipped (of the
                                    same dst the first pair stands) */

/* Bytes of workspace mtp_cache_resize and mtp_cache_fork need for a table of num_rows rows
 * (num_pairs pairs need no more than that many rows); 0 for invalid arguments. */
size_t mtp_cache_workspace_size(int32_t num_rows, int32_t max_pages_per_seq);

/*
 * Set every row's length: seq_lens = new_lens.  Rows that shrink give their surplus pages back
 * (new length 0 frees the row), rows that grow are handed pages.  A row whose last, partly
 * filled page (at the smaller of the two lengths) is shared gets a copy of it first, in all
 * layers.  If the free pages (after what is given back) do not suffice, no page is handed out or
 * copied, MTP_CACHE_ERR_FULL is set and every row stays at the smaller of its two lengths.
 *  new_lens   device int32 [num_rows], apart from seq_lens (else MTPATTN_E_ARG); a row to be left
 *             alone gets its own length.
 *  workspace  device, >= mtp_cache_workspace_size(num_rows, ..) bytes, 256-byte aligned, not
 *             initialised; calls that overlap on the GPU must use different ones.
 * A table entry outside [0, num_pages) that would be given back sets MTPATTN_ERR_PAGE and is
 * only cleared.  Two kernels are launched.
 */
int mtp_cache_resize(void* k_cache, void* v_cache, int32_t num_layers, int64_t layer_stride,
                     int64_t num_pages, int32_t num_kv_heads, int32_t* block_tables,
                     int32_t max_pages_per_seq, int32_t* seq_lens, int32_t num_rows,
                     int32_t* ref_counts, const int32_t* new_lens, void* workspace,
                     size_t workspace_bytes, int32_t* status, void* stream);

/*
 * Fork rows: row dst[i] (empty: length 0) becomes a copy of row src[i].  Full pages are shared
 * (their counts go up), a partly filled last page is copied into a new page in all layers.
 * Lengths are those at the start of the call.  If the free pages do not suffice for all pairs,
 * nothing is changed and MTP_CACHE_ERR_FULL is set.  A source row with a table entry outside
 * [0, num_pages) sets MTPATTN_ERR_PAGE and its pair is skipped.
 *  src, dst   device int32 [num_pairs], num_pairs <= num_rows.
 *  workspace  as in mtp_cache_resize.
 * Two kernels are launched.
 */
int mtp_cache_fork(void* k_cache, void* v_cache, int32_t num_layers, int64_t layer_stride,
                   int64_t num_pages, int32_t num_kv_heads, int32_t* block_tables,
                   int32_t max_pages_per_seq, int32_t* seq_lens, int32_t num_rows,
                   int32_t* ref_counts, const int32_t* src, const int32_t* dst,
                   int32_t num_pairs, void* workspace, size_t workspace_bytes, int32_t* status,
                   void* stream);

/*
 * Copy pages in all layers: page dst_pages[i] gets the contents of page src_pages[i].  A pair
 * with a page outside [0, num_pages) sets MTPATTN_ERR_PAGE and is skipped.  The destinations
 * must differ from one another and from the sources (else their contents are unspecified).
 *  src_pages, dst_pages  device int32 [num_pairs].
 * One kernel is launched.
 */
int mtp_cache_copy_pages(void* k_cache, void* v_cache, int32_t num_layers, int64_t layer_stride,
                         int64_t num_pages, int32_t num_kv_heads, const int32_t* src_pages,
                         const int32_t* dst_pages, int32_t num_pairs, int32_t* status,
                         void* stream);

/*
 * Keep the accepted path of each sequence's draft tree: with start_b = seq_lens[b] - n_b
 * (n_b = cu_seqlens_q[b+1] - cu_seqlens_q[b] nodes, 1 .. 64, see mtp_tree.h) the keys and values
 * of node accept_index[b][j] move to position start_b + j for j = 0 .. accept_len[b], in all
 * layers, in place, and new_seq_lens[b] = start_b + accept_len[b] + 1.  Pages are not given back
 * (mtp_cache_resize to new_seq_lens does that).  The pages that hold the tree must belong to
 * their row alone.
 *  accept_index device int32 [num_seqs][max_path] and accept_len [num_seqs], as the verification
 *               entry points of mtp_tree.h write them: accept_index[b][0] = 0, ascending.
 *  new_seq_lens device int32 [num_seqs], apart from all inputs (else MTPATTN_E_ARG).
 * A sequence whose path is not strictly ascending from 0 within its n_b nodes (or accept_len -1)
 * sets MTP_CACHE_ERR_LEN, one with a bad node count or length MTPATTN_ERR_QLEN, _QLEN_GT_SEQ or
 * _SEQ_TOO_LONG, one with a table entry outside [0, num_pages) under its tree MTPATTN_ERR_PAGE;
 * nothing of it is moved and its new length is its old one.  One kernel is launched.
 */
int mtp_cache_compact(void* k_cache, void* v_cache, int32_t num_layers, int64_t layer_stride,
                      int64_t num_pages, int32_t num_kv_heads, const int32_t* block_tables,
                      int32_t max_pages_per_seq, const int32_t* seq_lens,
                      const int32_t* cu_seqlens_q, int32_t num_seqs, int32_t total_q,
                      const int32_t* accept_index, const int32_t* accept_len, int32_t max_path,
                      int32_t* new_seq_lens, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MTP_CACHE_H */
