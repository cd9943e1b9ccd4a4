/*
 * mtp_rope.h — C ABI of the calls in libmtpattn.so (GB300, sm_103a) that make what the attention
 * calls read: rotary positions, rounding to e4m3, and the way of new tokens into the paged caches.
 *
 *   mtp_rope_append         q, k, v of new tokens: q rotated; k (rotated) and v into the paged K/V
 *                           cache of mtpattn.h, mtp_tree.h and mtp_cache.h;
 *   mtp_rope_latent_append  the same for the cache of latent vectors of mtp_latent.h;
 *   mtp_rope_prefill        the e4m3 operands of fmha_fwd_fp8_varlen (fmha_fp8_varlen.h) from the
 *                           projections' outputs.
 *
 * Rotary positions.  A rotated part of rot_dim elements (a multiple of 16) is rot_dim / 2 pairs; pair
 * i of a token at position m becomes
 *   (a, b) -> mscale * (a cos t - b sin t, b cos t + a sin t),   t = m * inv_freq[i].
 * The pair's elements are 2i and 2i + 1 of the part (interleaved != 0) or i and i + rot_dim / 2
 * (interleaved = 0, the half layout).  The angles are given as whole numbers of 2^-64 turns a
 * position, freqs[i] = round(2^64 * inv_freq[i] / (2 pi)) (mtp_rope_freqs makes them), so that
 * m * freqs[i] modulo 2^64 is the angle modulo one turn for every 32-bit position, without loss: far
 * positions are as exact as near ones.  Scaling for long contexts is in inv_freq and mscale.  A
 * negative position turns the other way.  Sines, cosines and the products are in float32.
 *
 * Codes.  code = e4m3(x * (1 / descale)) in float32, to nearest, ties to even; values beyond 448 (infinite
 * ones too) become +-448, NaN stays NaN (code 0x7f).  (The product, not the quotient: it may lie one
 * float32 step beside it, which changes a code only where the quotient lies on the border of two.)
 * descale is the number that the attention call is given.
 *
 * Inputs are of `dtype` (MTP_F32, MTP_BF16 or MTP_F16 of mtp_tree.h, all of a call the same), 16-byte
 * aligned, with unit stride along the head and strides (in elements) that are multiples of 8; strides
 * of heads may be those of a larger buffer (the output of a joint projection).
 *
 * Conventions are those of mtpattn.h: device pointers of the current device, no allocation, no
 * synchronisation, nothing read back (graph-capture safe), status codes MTPATTN_*, nothing launched on
 * an error return, device-side bits OR-ed into the optional status word.  One kernel is launched.
 * Results are the same bits in every call with the same arguments.
 */
#ifndef MTP_ROPE_H
#define MTP_ROPE_H

#include <stddef.h>
#include <stdint.h>

#include "mtpattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* freqs[i] = round(2^64 * inv_freq[i] / (2 pi)) mod 2^64, on the host: inv_freq and freqs are host
 * arrays of n.  MTPATTN_E_ARG for a null pointer, n < 0, or an inv_freq that is negative, not finite or
 * above 2^20. */
int mtp_rope_freqs(const double* inv_freq, int32_t n, int64_t* freqs);

/*
 * New tokens into the K/V cache.  Sequence b's n_b = cu_seqlens_q[b+1] - cu_seqlens_q[b] tokens (any
 * number from 0, packed at rows cu_seqlens_q[b] ..) are the last n_b of its seq_lens[b] tokens: row
 * cu_seqlens_q[b] + i goes to place seq_lens[b] - n_b + i, page block_tables[b][place / 16].  (A token's
 * position is given apart from its place: in a draft tree it goes by depth.)
 *  q            device [total_q][num_q_heads][256], or NULL with num_q_heads = 0: no q
 *  k, v         device [total_q][num_kv_heads][256]
 *  positions    device int32 [total_q]
 *  freqs        device int64 [rot_dim / 2], 8-byte aligned; NULL with rot_dim = 0
 *  rot_dim      0 (nothing is rotated) or a multiple of 16 up to 256: the first elements of a head of
 *               q and k
 *  k_cache, v_cache, num_pages, block_tables, max_pages_per_seq, seq_lens, cu_seqlens_q
 *               as in mtp_verify_attn_fwd; the pages under the new tokens belong to their row alone
 *  k_descale, v_descale   device float32, one element each
 *  q_out        device bf16 [total_q][num_q_heads][256], strides as the inputs'.  q itself, if that is
 *               bf16, with q's strides; else apart from all inputs.  Its rows are apart from one another.
 * Rows that belong to no sequence (before cu_seqlens_q[0], behind the last) are not written anywhere.
 * A sequence with more tokens than seq_lens[b] (MTPATTN_ERR_QLEN_GT_SEQ) or more than its table holds
 * (_SEQ_TOO_LONG), and a token whose page is outside [0, num_pages) (_PAGE), are left out of the caches;
 * their q is rotated all the same.  Where cu_seqlens_q does not ascend, or leaves 0 .. total_q,
 * MTPATTN_ERR_QLEN is set: then a row is known if one sequence alone, whose own two entries ascend within
 * total_q, claims it, and other rows are not written anywhere.
 */
int mtp_rope_append(const void* q, int64_t q_stride_tok, int64_t q_stride_head, const void* k,
                    int64_t k_stride_tok, int64_t k_stride_head, const void* v, int64_t v_stride_tok,
                    int64_t v_stride_head, int32_t dtype, const int32_t* positions,
                    const int64_t* freqs, int32_t rot_dim, int32_t interleaved, float mscale,
                    void* k_cache, void* v_cache, int64_t num_pages, const int32_t* block_tables,
                    int32_t max_pages_per_seq, const int32_t* seq_lens, const int32_t* cu_seqlens_q,
                    int32_t num_seqs, int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads,
                    const float* k_descale, const float* v_descale, void* q_out,
                    int64_t q_out_stride_tok, int64_t q_out_stride_head, int32_t* status,
                    void* stream);

/*
 * New tokens into the latent cache of mtp_latent.h: a token's 576 codes are its latent vector (512, not
 * rotated) and its rotated part (64).
 *  q_rope       device [total_q][num_heads][64], or NULL with num_heads = 0
 *  latent       device [total_q][512], row stride latent_stride
 *  k_rope       device [total_q][64], row stride k_rope_stride
 *  freqs        device int64 [32]
 *  cache        device e4m3 [num_pages][16][576]
 *  descale      device float32, one element: of all 576 codes
 *  q_out        device bf16 [total_q][num_heads][64], strides in elements, multiples of 8: the end of
 *               the rows of 576 that mtp_latent_attn_fwd reads.  q_rope itself, if that is bf16, with its
 *               strides; else apart from all inputs.
 * All else as in mtp_rope_append.
 */
int mtp_rope_latent_append(const void* q_rope, int64_t q_stride_tok, int64_t q_stride_head,
                           const void* latent, int64_t latent_stride, const void* k_rope,
                           int64_t k_rope_stride, int32_t dtype, const int32_t* positions,
                           const int64_t* freqs, int32_t interleaved, float mscale, void* cache,
                           int64_t num_pages, const int32_t* block_tables, int32_t max_pages_per_seq,
                           const int32_t* seq_lens, const int32_t* cu_seqlens_q, int32_t num_seqs,
                           int32_t total_q, int32_t num_heads, const float* descale, void* q_out,
                           int64_t q_out_stride_tok, int64_t q_out_stride_head, int32_t* status,
                           void* stream);

/*
 * The prefill attention's operands (the expanded form of latent attention):
 *   q8[t][h] = e4m3 of q[t][h] with its last 64 elements rotated         (192 codes)
 *   k8[t][h] = e4m3 of k[t][h] (128), then of k_rope[t] (64), rotated     (192 codes)
 *   v8[t][h] = e4m3 of v[t][h]                                            (128 codes)
 *  q            device [total][num_q_heads][192]
 *  k, v         device [total][num_kv_heads][128]
 *  k_rope       device [total][64], row stride k_rope_stride: shared by all heads
 *  positions    device int32 [total]; freqs device int64 [32]
 *  q8, k8, v8   device e4m3, contiguous [total][heads][192, 192, 128], 16-byte aligned, apart from all
 *               inputs and one another
 * num_q_heads is a multiple of num_kv_heads.
 */
int mtp_rope_prefill(const void* q, int64_t q_stride_tok, int64_t q_stride_head, const void* k,
                     int64_t k_stride_tok, int64_t k_stride_head, const void* k_rope,
                     int64_t k_rope_stride, const void* v, int64_t v_stride_tok,
                     int64_t v_stride_head, int32_t dtype, const int32_t* positions,
                     const int64_t* freqs, int32_t interleaved, float mscale, int32_t total,
                     int32_t num_q_heads, int32_t num_kv_heads, const float* q_descale,
                     const float* k_descale, const float* v_descale, void* q8, void* k8, void* v8,
                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MTP_ROPE_H */
