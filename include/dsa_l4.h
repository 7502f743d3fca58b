/*
 * dsa_l4.h - the 4-bit latent cache of the DSA step, the attention weight its
 * tokens receive, and the eviction of tokens by it (NVIDIA B200, sm_100a).
 *
 * The conventions of dsa.h hold throughout: caller-owned device memory, calls
 * asynchronous on `stream` (NULL: the per-thread default stream), host checks
 * before any launch with no side effects on refusal, device-side range checks
 * that skip the access and are read back with dsa_workspace_check(), and a
 * workspace that serves one call at a time.  A block table has at most
 * 2^25 - 1 pages per sequence (DSA_ERR_UNSUPPORTED).
 *
 * Row format ("l4")
 * -----------------
 * A latent row of W = R + P columns stands for
 *     L[c] = 2^e * s[c / 16] * v[c]
 * with v[c] an e2m1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives),
 * s[.] one E4M3 scale per block of 16 columns and 2^e one power of two per
 * token.  It is stored in dsa_l4_row_bytes(R, P) bytes (336 at W = 576, against
 * 1,152 in bf16 and 580 in E4M3):
 *     bytes [0, W/2)            codes: sign, 2 exponent bits, 1 mantissa bit;
 *                               the even column of a pair in the low nibble
 *     bytes [W/2, W/2 + W/16)   block scales, E4M3, finite and not negative
 *     byte  W/2 + W/16          e + 127, with e in [-60, 60]
 *     up to a multiple of 16    zero
 * and serves as key (all W columns) and value (the first R), as a bf16 row does.
 * Every such value has at most 6 significant bits: it is exact in bf16, and
 * s * v is exact in fp16, which is what the kernels multiply.
 *   latent4_pages [num_pages, 64, dsa_l4_row_bytes] uint8, 16-byte aligned
 * The pages hold weights in INT4 and FP8 with scales per block ("GLM on an
 * A100, in Vx", section "INT4, FP8 and BF16"); a 4-bit cache and eviction have
 * no counterpart there.
 */
#ifndef DSA_L4_H_
#define DSA_L4_H_

#include "dsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Operation ids for dsa_l4_workspace_bytes(). */
typedef enum {
  DSA_L4_OP_STATUS = 0, /* dsa_cache_append_l4, dsa_cache_read_l4: the status block */
  DSA_L4_OP_SPARSE_MLA = 1,        /* dsa_sparse_mla_decode_l4 / _prefill_l4 */
  DSA_L4_OP_ATTENTION_FORWARD = 2, /* dsa_attention_forward_l4               */
  DSA_L4_OP_ATTENTION_MASS = 3,    /* dsa_attention_mass / _l8 / _l4          */
  DSA_L4_OP_CACHE_EVICT = 4        /* dsa_cache_evict                         */
} dsa_l4_op_t;

/* Bytes of one stored row; 0 when R or P is outside what the kernels take
 * (R a multiple of 64 up to 512, P a multiple of 16, R + P <= 576). */
DSA_API size_t dsa_l4_row_bytes(int32_t R, int32_t P);

/* Bytes of workspace `op` needs for these dims and cache (dsa_workspace_init
 * clears its status block, dsa_workspace_check reads it).  Returns 0 for
 * invalid input.  dims may be NULL for DSA_L4_OP_CACHE_EVICT, which depends on
 * the cache alone. */
DSA_API size_t dsa_l4_workspace_bytes(dsa_l4_op_t op, const dsa_dims_t *dims,
                                      const dsa_cache_t *cache);

/* Append: the new tokens' index keys (bf16, as dsa_cache_append) and latent
 * rows, the latter quantised, into the paged caches.
 *   k_idx_new [n_q, D_I] bf16, latent_new [n_q, R + P] bf16, 16-byte aligned
 * A row x is stored with the least e for which max|x| <= 2688 * 2^e (clamped to
 * [-60, 60]; 0 for a row of zeros), s[b] = E4M3(max|x_b| / (6 * 2^e)) and
 * v = e2m1(x / (s[b] * 2^e)), both rounded to nearest, ties to even, and
 * saturating (an infinity is stored as the largest value its row's scales
 * allow; a NaN as some finite value).  A block whose scale rounds to zero is
 * stored as zeros.  Positions, page checks and the use of dims as in
 * dsa_cache_append; distinct rows must target distinct slots.  Workspace:
 * DSA_L4_OP_STATUS. */
DSA_API dsa_status_t dsa_cache_append_l4(const uint16_t *k_idx_new, const uint16_t *latent_new,
                                 uint16_t *k_idx_pages, uint8_t *latent4_pages,
                                 const dsa_cache_t *cache, const dsa_dims_t *dims, void *ws,
                                 size_t ws_bytes, dsa_stream_t stream);

/* Read back: the values of stored rows, exactly, as bf16.
 *   idx   [n_q, topk] int32 token positions, in any order; row r's belong to
 *         sequence r (dims.causal == 0) or 0 (dims.causal == 1).  -1 gives a
 *         row of zeros; a position outside the row's context is flagged and
 *         gives a row of zeros too
 *   rows  [n_q, topk, R + P] bf16 output, 16-byte aligned
 * Workspace: DSA_L4_OP_STATUS. */
DSA_API dsa_status_t dsa_cache_read_l4(const uint8_t *latent4_pages, const dsa_cache_t *cache,
                               const int32_t *idx, const dsa_dims_t *dims, uint16_t *rows,
                               void *ws, size_t ws_bytes, dsa_stream_t stream);

/* Sparse MLA over a 4-bit latent cache: dsa_sparse_mla_decode / _prefill with
 * the rows of the format above (everything else as there: -1 slots, positions
 * outside the context skipped and flagged, rows that keep nothing get out = 0
 * and lse = -inf).  Products and weights: the stored rows enter the tensor
 * cores exactly; q enters as fp16 after a power-of-two scale per query row, so
 * a q element is carried exactly unless it is below 2^-28 of the row's largest
 * magnitude (then to 2^-39 of it); the softmax weights enter as two fp16 terms
 * (22 bits), and what a token adds to out is lost below 2^-31 of the row's
 * largest such product; sums are fp32, which the tensor cores truncate rather
 * than round: against float64, out is off by up to 2e-6 of its largest magnitude
 * at 32 rows of 2,048 kept tokens, 4e-6 where one CTA takes 1,024 or more (columns
 * from 256 on, whose two terms share a sum, about twice what the others are), and
 * lse by 2e-6.  q must be finite.
 * Workspace: DSA_L4_OP_SPARSE_MLA. */
DSA_API dsa_status_t dsa_sparse_mla_decode_l4(const uint16_t *q, const uint8_t *latent4_pages,
                                      const dsa_cache_t *cache, const int32_t *idx,
                                      const dsa_dims_t *dims, float *out, float *lse, void *ws,
                                      size_t ws_bytes, dsa_stream_t stream);
DSA_API dsa_status_t dsa_sparse_mla_prefill_l4(const uint16_t *q, const uint8_t *latent4_pages,
                                       const dsa_cache_t *cache, const int32_t *idx,
                                       const dsa_dims_t *dims, float *out, float *lse, void *ws,
                                       size_t ws_bytes, dsa_stream_t stream);

/* The whole step over bf16 index keys and a 4-bit latent cache: indexer scores
 * -> exact top-k -> dsa_sparse_mla_*_l4, one call (as dsa_attention_forward).
 * Workspace: DSA_L4_OP_ATTENTION_FORWARD. */
DSA_API dsa_status_t dsa_attention_forward_l4(const uint16_t *q_idx, const float *w,
                                      const uint16_t *k_idx_pages, const uint16_t *q,
                                      const uint8_t *latent4_pages, const dsa_cache_t *cache,
                                      const dsa_dims_t *dims, int32_t *idx_out, float *out,
                                      float *lse, void *ws, size_t ws_bytes, dsa_stream_t stream);

/* Accumulated attention weight: what the step's softmax gave each cached
 * token, summed over heads (and over the rows of a causal chunk), added to a
 * running sum per token.
 *   mass_out[b, s] = decay * mass_in[b, s] + sum_{r of b, h, j: idx[r,j] = s} exp(z[r,h,j] - lse[r,h])
 *   z[r,h,j] = scale * q[r,h] . L[idx[r,j]]
 *   q, idx    the step's query and kept positions, as in dsa_sparse_mla_decode
 *             / _prefill (dims.causal selects which; unused slots -1; a
 *             position outside the row's context is skipped and flagged)
 *   lse       [n_q, H] fp32, the step's; a row with lse = -inf adds nothing
 *   decay     finite, >= 0
 *   mass_in   [num_seqs, mass_ld] fp32, or NULL for zeros.  Every entry s < len(b)
 *             is read: a token that was appended since the sums were last written
 *             has to hold 0 there.  Neither an append nor an eviction clears it,
 *             so a buffer that held a longer sequence before an eviction still
 *             holds the sums of tokens that are gone
 *   mass_out  [num_seqs, mass_ld] fp32; may be mass_in, else apart from it.  Entries s < len(b) are
 *             written (len(b): seq_lens[b], at most max_seq_len; for a causal
 *             chunk q_pos0 + n_q); entries past that are left untouched, and
 *             so is everything when n_q = 0.  mass_ld >= max_seq_len, for a
 *             causal chunk >= q_pos0 + n_q (which is sequence 0: only row 0
 *             is written)
 * A position that a row holds twice counts twice.  Causal chunks add their
 * rows in 64-bit fixed point, so the result does not depend on the order in
 * which the rows ran (a NaN weight, and one of 128 or more, which no lse of the
 * step's leaves, is added in fp32 instead).  A step is n_q 2^-56, n_q rounded up
 * to a power of two (2^-47 for 512 rows); a weight below half of it adds nothing.
 * A decode row adds in fp32, once per place.  Against float64, with the lse given, a mass is off
 * by about 1e-6 of the largest (its logits are tensor-core sums as above).  Workspace: DSA_L4_OP_ATTENTION_MASS.  The three forms differ in
 * the latent cache they read: bf16, E4M3 with one scale per token, 4-bit. */
DSA_API dsa_status_t dsa_attention_mass(const uint16_t *q, const uint16_t *latent_pages,
                                const dsa_cache_t *cache, const int32_t *idx, const float *lse,
                                const dsa_dims_t *dims, float decay, const float *mass_in,
                                float *mass_out, int64_t mass_ld, void *ws, size_t ws_bytes,
                                dsa_stream_t stream);
DSA_API dsa_status_t dsa_attention_mass_l8(const uint16_t *q, const uint8_t *latent8_pages,
                                   const float *latent_scale, const dsa_cache_t *cache,
                                   const int32_t *idx, const float *lse, const dsa_dims_t *dims,
                                   float decay, const float *mass_in, float *mass_out,
                                   int64_t mass_ld, void *ws, size_t ws_bytes,
                                   dsa_stream_t stream);
DSA_API dsa_status_t dsa_attention_mass_l4(const uint16_t *q, const uint8_t *latent4_pages,
                                   const dsa_cache_t *cache, const int32_t *idx, const float *lse,
                                   const dsa_dims_t *dims, float decay, const float *mass_in,
                                   float *mass_out, int64_t mass_ld, void *ws, size_t ws_bytes,
                                   dsa_stream_t stream);

/* One paged pool that an eviction moves: rows of row_bytes bytes, a multiple
 * of 4 up to 4,096, one per token, pool row = page * 64 + slot.  src is indexed
 * by the cache's block table, dst by the destination's.  Both are 16-byte
 * aligned when row_bytes is a multiple of 16, else 4-byte aligned.  src and
 * dst may be the same pool as long as the source and destination pages of the
 * call are disjoint. */
typedef struct {
  const void *src;
  void *dst;
  int32_t row_bytes;
} dsa_pool_t;

#define DSA_EVICT_MAX_POOLS 4

/* Which tokens an eviction keeps, and where they go. */
typedef struct {
  int32_t budget;   /* tokens kept of a longer sequence, >= 1                    */
  int32_t sinks;    /* the first `sinks` tokens are always kept, >= 0            */
  int32_t recent;   /* the last `recent` tokens are always kept, >= 0;
                       sinks + recent <= budget                                  */
  const int32_t *dst_block_table; /* [num_seqs, dst_max_pages] destination pages */
  int32_t dst_max_pages;          /* dst_max_pages * 64 >= min(budget, max_seq_len) */
  int32_t dst_num_pages;          /* pages in each destination pool (device check) */
} dsa_evict_t;

/* Eviction: every sequence keeps min(budget, len) tokens - its first `sinks`,
 * its last `recent`, and of the others those with the largest mass, the lower
 * position winning ties (a NaN ranks as -inf, +inf as the largest finite
 * value) - and their rows of
 * all pools, and their masses, are compacted into destination pages in their
 * old order.  Token i of the result lives in page dst_block_table[b, i / 64],
 * slot i % 64; the latent rows keep the rotary positions they were written
 * with.
 *   pools     [n_pools] (host array, 0 <= n_pools <= DSA_EVICT_MAX_POOLS)
 *   cache     the source: seq_lens, block_table, num_pages, max_seq_len (a
 *             length above max_seq_len counts as max_seq_len)
 *   mass      [num_seqs, mass_ld] fp32, mass_ld >= max_seq_len
 *   mass_dst  [num_seqs, mass_dst_ld] fp32, mass_dst_ld >= min(budget,
 *             max_seq_len); may be NULL; must not overlap mass (mass itself
 *             is refused)
 *   new_lens  [num_seqs] int32 output; may be cache->seq_lens
 *   kept      [num_seqs, budget] int32 output: the kept positions, ascending,
 *             -1 padded; may be NULL
 * Destination rows, masses and pages past new_lens[b] are left untouched: set
 * mass_dst[b, s] to 0 before dsa_attention_mass reads it for a new token s.  A
 * source or destination page id out of range skips that row and is reported
 * as DSA_ERR_DEVICE_CHECK.  Workspace: DSA_L4_OP_CACHE_EVICT. */
DSA_API dsa_status_t dsa_cache_evict(const dsa_pool_t *pools, int32_t n_pools,
                             const dsa_cache_t *cache, const dsa_evict_t *evict,
                             const float *mass, int64_t mass_ld, float *mass_dst,
                             int64_t mass_dst_ld, int32_t *new_lens, int32_t *kept, void *ws,
                             size_t ws_bytes, dsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_L4_H_ */
