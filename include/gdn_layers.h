/*
 * gdn_layers.h -- C ABI of the operators that stand around the delta-rule
 * operators of gdn.h in a hybrid model: the norm in front of each layer and on
 * the delta rule's own output, and the softmax-attention layer that such models
 * put beside every few delta-rule layers (rotary positions, a paged key/value
 * cache, and one decode step over it).
 *
 *   gdn_rms_norm        root-mean-square norm with the residual's addition, the
 *                       SiLU gate of the delta rule's output and an 8-bit output
 *   gdn_rope_fwd        rotary positions of q and k, with k and v written into
 *                       a paged cache
 *   gdn_paged_attn_fwd  attention of one new token per sequence over that cache
 *
 * Conventions (device pointers, dense row-major tensors, asynchronous on
 * `stream`, status codes, the dtype codes GDN_DTYPE_*) are those of gdn.h.
 * Every call runs on the calling thread's current device, which `stream` must
 * belong to.  Argument errors are returned before anything is enqueued.  All
 * calls may be captured into a CUDA graph.
 */
#ifndef GDN_LAYERS_H_
#define GDN_LAYERS_H_

#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* output form of gdn_rms_norm */
#define GDN_QUANT_NONE 0  /* out in act_dtype                                     */
#define GDN_QUANT_ROW 1   /* out in e4m3, one fp32 scale per row                  */
#define GDN_QUANT_BLOCK 2 /* out in e4m3, one fp32 scale per row and GDN_QUANT_GROUP columns */
#define GDN_QUANT_GROUP 128
#define GDN_NORM_MAX_WIDTH 32768
#define GDN_ROPE_MAX_DIM 256

/*
 * gdn_rms_norm -- root-mean-square norm of each row.
 *
 *     z = x + residual                      (z = x without a residual)
 *     y = z / sqrt(mean(z^2) + eps) * (weight + weight_offset)
 *     y = y * gate / (1 + e^-gate)          (with a gate)
 *     residual_out = z, rounded to act_dtype
 *     out = y, rounded to act_dtype, or in 8 bits:
 *       scale = max(max |y| / 448, 2^-126) over the row (GDN_QUANT_ROW) or over
 *       each GDN_QUANT_GROUP columns of it (GDN_QUANT_BLOCK; the last group of a
 *       row may be shorter), out = y / scale rounded to nearest e4m3, so that
 *       y is about out * scale
 *
 * z, the mean and y are fp32; y is computed from z before z is rounded.  With
 * rows = T Nv and width = Dv this is the gated norm of a delta-rule layer's
 * output [T, Nv, Dv].  weight_offset = 1 takes weights stored around zero.
 *
 *   x             [rows, width] of act_dtype
 *   residual      [rows, width] of act_dtype, or NULL; needs residual_out
 *   gate          [rows, width] of act_dtype, or NULL
 *   weight        [width] of weight_dtype, which is act_dtype or fp32
 *   out           [rows, width] of act_dtype, or e4m3 bytes; may be x itself
 *                 when quant is GDN_QUANT_NONE
 *   residual_out  [rows, width] of act_dtype; may be residual itself
 *   scales        fp32 [rows] or [rows, ceil(width / GDN_QUANT_GROUP)]; NULL
 *                 without an 8-bit output
 *   rows          >= 0 (0 is a no-op); width 1 .. GDN_NORM_MAX_WIDTH, at most
 *                 GDN_NORM_MAX_WIDTH - 8 where it is no multiple of 8
 * A row that holds a NaN or an infinity in z comes out as NaN where the formula
 * gives NaN.  Where the sum of a row's z^2 is beyond fp32 (3.4e38: |z| of 1.8e19,
 * or of 1e17 in each of 32768 columns) the row comes out as zero.  Below a gate
 * of -87 the factor gate / (1 + e^-gate), under 2e-36, is zero.
 * Alignment: 16 bytes for the matrices and weight, 4 for scales.  Errors:
 * GDN_ERR_NULL_ARG, GDN_ERR_BAD_SHAPE (sizes, unknown codes), GDN_ERR_UNSUPPORTED
 * (width, rows > 2^31 - 32), GDN_ERR_ALIGNMENT, GDN_ERR_OVERLAP (an output on an
 * input or on another output, beyond the two cases above), GDN_ERR_CUDA.
 */
int gdn_rms_norm(const void *x, const void *residual, const void *gate, const void *weight, float eps,
                 float weight_offset, void *out, void *residual_out, float *scales, int64_t rows, int32_t width,
                 int32_t act_dtype, int32_t weight_dtype, int32_t quant, void *stream);

/*
 * gdn_rope_fwd -- rotary positions of the queries and keys, and the write of
 * the new keys and values into a paged cache.
 *
 * Token t at position p turns the first `rotary` columns of each head of q and
 * k by the angles p inv_freq[i], i < n = rotary / 2:
 *     (a, b) -> mscale (a cos - b sin, b cos + a sin)
 * where (a, b) are the columns (i, n + i), or (2 i, 2 i + 1) when interleaved.
 * The other columns pass unchanged.  The angle is the product of position and
 * inv_freq in 64 bits, reduced in 64 bits, so it is as good at position 2^31 as
 * near zero (|angle| below 2^50).  Its sine and cosine are within 2^-21 of the
 * exact ones for 16-bit activations, within 2^-24 for fp32.
 *
 *   q             [T, Hq, D] of act_dtype; k [T, Hkv, D]
 *   v             [T, Hkv, D], or NULL without a cache
 *   positions     int32 [T]
 *   inv_freq      fp32 [rotary / 2], with any scaling for long contexts in it
 *   slots         int32 [T]: cache row (page * page_size + place in the page) of
 *                 each token.  A slot outside [0, cache_rows) marks padding: its
 *                 token is not written.  Slots in one call have to differ, else
 *                 the row that two tokens share holds either's elements
 *   q_out         [T, Hq, D]; may be q itself
 *   k_out         [T, Hkv, D], the turned keys, or NULL (then a cache is
 *                 needed); may be k itself
 *   k_cache, v_cache   [cache_rows, Hkv, D] of act_dtype (the pages of
 *                 gdn_paged_attn_fwd in a row), or both NULL.  Rows that no slot
 *                 names are left as they were
 *   T             >= 0 (0 is a no-op); Hq, Hkv >= 1; D a multiple of 8 up to
 *                 GDN_ROPE_MAX_DIM; rotary even, 0 .. D
 * Alignment: 16 bytes for q, k, v, q_out, k_out and the caches, 4 for the rest.
 * Errors: GDN_ERR_NULL_ARG, GDN_ERR_BAD_SHAPE, GDN_ERR_UNSUPPORTED (D, T >= 2^31,
 * cache_rows >= 2^31, more than 65535 heads), GDN_ERR_ALIGNMENT, GDN_ERR_OVERLAP, GDN_ERR_CUDA.
 */
int gdn_rope_fwd(const void *q, const void *k, const void *v, const int32_t *positions, const float *inv_freq,
                 const int32_t *slots, float mscale, void *q_out, void *k_out, void *k_cache, void *v_cache,
                 int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t rotary, int32_t interleaved,
                 int64_t cache_rows, int32_t act_dtype, void *stream);

/*
 * gdn_paged_attn_fwd -- attention of one new token of each sequence over a
 * paged key/value cache.
 *
 *     s_j = scale q . k_j,  p = softmax(s),  out = sum_j p_j v_j,  lse = log sum_j e^s_j
 * over the seq_lens[b] keys of sequence b, the new token's own among them (it
 * is written first, see gdn_rope_fwd).  The cache is read once for each 16 query
 * heads of a key/value head.  Query head h reads key/value head
 * h / (Hq / Hkv).  Token j of sequence b lies on page block_table[b][j /
 * page_size], at place j % page_size.  Several new tokens of one sequence
 * (speculative decoding) are as many rows with the same pages and growing
 * lengths.
 *
 *   q             [B, Hq, D] of act_dtype (bf16 or fp16)
 *   k_cache, v_cache   [P, page_size, Hkv, D] of act_dtype
 *   block_table   int32 [B, max_pages]; entries past a sequence's last page are
 *                 not read
 *   seq_lens      int32 [B], 0 .. max_pages * page_size.  A length of 0 gives a
 *                 zero row and lse = -infinity
 *   scale         <= 0 selects 1/sqrt(D); else up to 2.3e38 (NaN and infinity
 *                 are GDN_ERR_BAD_SHAPE)
 *   out           [B, Hq, D] of act_dtype; lse fp32 [B, Hq] or NULL
 *   max_seqlen    the longest sequence if known, else 0: keeps the grid and the
 *                 workspace of a small call small; any value gives a right result
 *   D             64, 128 or 256; Hq a multiple of Hkv; page_size >= 1
 *   workspace     >= gdn_paged_attn_workspace_bytes(...) for the same sizes and
 *                 max_seqlen, 16-byte aligned, or NULL: the call then allocates
 *                 and frees it stream-ordered.  Calls that may overlap on the
 *                 GPU (two captured graphs among them) need workspaces of their own
 * A sequence with a length outside its range or a page outside [0, P) among its
 * pages reads nothing out of bounds and comes out as NaN (out and lse), the
 * others are not affected.  NaN and infinities in a sequence's own rows come out
 * as NaN where the formula gives NaN, but for a sequence whose every score is
 * -infinity: it comes out as one without keys (a zero row, lse = -infinity).  An
 * infinity in v comes out as an infinity or NaN (p is
 * multiplied in two parts, the second of either sign); cache rows that no sequence lists are never read.
 * A key's weight is held to 16 bits or more, in fp16 of keys more than 16 nats below the row's largest score to 2^-40 of
 * the largest weight.
 * q . k is formed in fp32: up to 3.4e38 scores of any size give a right row, beyond it one is an infinity.
 * Alignment: 16 bytes for q, the caches, out and workspace, 4 for the rest.  Errors:
 * GDN_ERR_NULL_ARG, GDN_ERR_BAD_SHAPE, GDN_ERR_UNSUPPORTED (act_dtype, D, P *
 * page_size >= 2^31, max_pages * page_size > 2^30, B >= 2^30, Hq > 65535), GDN_ERR_ALIGNMENT,
 * GDN_ERR_WORKSPACE, GDN_ERR_OVERLAP, GDN_ERR_CUDA.  B == 0 is a no-op.
 */
size_t gdn_paged_attn_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                                      int32_t max_pages, int32_t max_seqlen);
int gdn_paged_attn_fwd(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                       const int32_t *seq_lens, float scale, void *out, float *lse, int32_t B, int32_t Hq,
                       int32_t Hkv, int32_t D, int32_t P, int32_t page_size, int32_t max_pages, int32_t max_seqlen,
                       int32_t act_dtype, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LAYERS_H_ */
