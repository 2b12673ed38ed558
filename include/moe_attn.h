/*
 * moe_attn.h - gated grouped-head attention over a paged key-value cache (the
 * layers between the linear-attention ones, see moe_gdn.h).
 *
 * One quarter of the layers of the models this library serves keeps a growing
 * cache of keys and values (page "Show HN: Run an 80B Qwen in 4.3 GB of RAM on
 * a Mac and a 35B on an iPhone", how-it-works list; the validation paragraph
 * names gated GQA).  The pages give no formula; for token t of a sequence at
 * position p (counted from 0 over the whole sequence), query head h and its
 * key head hk = h / (q_heads / kv_heads):
 *
 *   o[t][h] = sigmoid(gate[t][h]) * sum_{j <= p} w_j v_j[hk]
 *   w_j     = exp(z_j) / sum_{i <= p} exp(z_i),   z_j = scale * q[t][h] . k_j[hk]
 *
 * (without a gate the factor is 1).  Before that, moe_kv_append brings the new
 * tokens' keys and values into the cache, with the RMS norms and the rotary
 * positions of queries and keys:
 *
 *   x^  = x / sqrt(mean(x^2) + eps) * norm           (x without a norm)
 *   x'_i        = x^_i cos(a_i) - x^_(i+r/2) sin(a_i)
 *   x'_(i+r/2)  = x^_(i+r/2) cos(a_i) + x^_i sin(a_i)    i < r/2, a_i = p * freq_i
 *   x'_i        = x^_i                                    i >= r = rot_dim
 *
 * The cache: n_pages pages of page_size tokens, k and v each
 *   [n_pages][kv_heads][page_size][head_dim] in act_dtype,
 * table [batch][max_pages] int32 (page i of sequence b holds its positions
 * i * page_size ..) and length [batch] int32, each sequence's tokens with the
 * new ones of the call included.  Sequences may share pages for reading;
 * positions that one call writes must lie on pages of their own.  A length is
 * read as the nearest of 0 and max_pages * page_size; positions whose table
 * entry names no page (outside [0, n_pages)) do not take part: nothing is
 * written there and no query sees them.  What lies behind a sequence's length,
 * or after a token's position, has no influence on that token's result,
 * whatever it holds.
 *
 * The tokens of a call: moe_attn_decode takes the last token of every sequence
 * (row b of q, gate and o).  The others take seq_off (device int32 [batch+1],
 * non-decreasing, within [0, n_tokens]): sequence b owns rows seq_off[b] ..
 * seq_off[b+1] - 1, its last n positions.  Offsets outside the range are read
 * as its nearest end, and an end before its start as no tokens: no access
 * leaves the buffers, but where offsets decrease the results are not defined.
 * Rows outside every sequence are left as they are.  A row that sees no
 * position (length 0, fewer positions than new tokens, no page that is one)
 * gives 0, whatever its gate is.
 *
 * Sums, maxima and the softmax's sums are fp32 in a fixed order (bitwise
 * repeatable); the split of a long sequence over workgroups depends on the
 * whole batch, so a token's results may differ in their last bits between
 * batches.  Softmax weights meet the values as act_dtype in moe_attn_prefill
 * (each off by up to half a step; their sum is that of the unrounded ones) and
 * as the sum of two such numbers in moe_attn_decode.  Each output is rounded
 * once to act_dtype.  A non-finite key or value makes the results of the tokens
 * that see it unusable (a score of -infinity counts as a weight of 0; a row with
 * no other gives 0), and so do products q . k or scores that leave fp32's range,
 * and values whose sum of magnitudes over the positions that a token sees does.
 * Scores so large that fp32 holds no digits behind their point still give means
 * of values.
 */
#ifndef MOE_AMD_MOE_ATTN_H
#define MOE_AMD_MOE_ATTN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* batch:     B in [0, 65535] (0 is a no-op)
 * kv_heads:  1..128
 * q_heads:   1 to 16 times kv_heads
 * head_dim:  64, 128 or 256
 * act_dtype: MOE_F16 or MOE_BF16 (cache, queries, gates, outputs)
 * page_size: 16, 32, 64, 128 or 256
 * n_pages:   >= 1
 * max_pages: >= 1, max_pages * page_size up to 2^30 and batch * kv_heads *
 *            max_pages * page_size up to 2^37
 * Calls that take n_tokens hold up to 2^22 blocks of 256 / (q_heads / kv_heads)
 * (rounded down) tokens: kv_heads * (n_tokens / block + batch), where a batch
 * above n_tokens counts as n_tokens. */
typedef struct {
  int32_t batch, q_heads, kv_heads, head_dim, act_dtype, page_size, n_pages, max_pages;
} moe_attn_desc;

/* Device buffers of the cache: k and v 16-byte, table and length 4-byte aligned. */
typedef struct {
  void *k, *v;
  const int32_t *table, *length;
} moe_kv_cache;

/* Rows of a call: head h of token t starts at data + t * token_stride + h *
 * head_stride (elements; both multiples of 8 in [0, 2^31)) and is head_dim values
 * long; 16-byte aligned.  So a slice of a wider projection's output can be
 * taken as it is. */
typedef struct {
  const void* data;
  int64_t token_stride, head_stride;
} moe_attn_rows;

/* Writes the n_tokens (up to 2^20) new tokens' keys and values into the cache;
 * seq_off NULL: one token for each sequence (n_tokens == batch).  With q, also
 * writes q_out [n_tokens][q_heads][head_dim] (16-byte aligned; q itself where q
 * lies like that).  Norms (device fp32 [head_dim], 16-byte aligned) and freq
 * (device fp64 [rot_dim / 2], radians per position) may be NULL; rot_dim: a
 * multiple of 16 up to head_dim (0: none).  v is copied.  Arithmetic is fp32 (the angles fp64) and
 * each value is rounded once; a row whose sum of squares overflows fp32 counts
 * as zero.  Tokens without a position (more new tokens than the length) are
 * left out, their rows of q_out included. */
moe_status moe_kv_append(const moe_attn_desc* desc, const moe_kv_cache* cache, const int32_t* seq_off_or_null,
                         int32_t n_tokens, const moe_attn_rows* k, const moe_attn_rows* v,
                         const moe_attn_rows* q_or_null, void* q_out_or_null, const float* q_norm_or_null,
                         const float* k_norm_or_null, float eps, const double* freq_or_null, int32_t rot_dim,
                         moe_stream stream);

/* Bytes of workspace (256-byte aligned) that moe_attn_decode (n_tokens 0) and
 * moe_attn_prefill of up to n_tokens tokens need: up to 9 MB for the one, up to
 * 137 MB for the other.  The workspace is only used while a call runs. */
moe_status moe_attn_workspace_bytes(const moe_attn_desc* desc, int32_t n_tokens, size_t* bytes);

/* Attention of the last token of every sequence: q, gate rows [batch], o
 * [batch][q_heads][head_dim] (16-byte aligned).  scale: finite, up to 2^127 either way. */
moe_status moe_attn_decode(const moe_attn_desc* desc, const moe_kv_cache* cache, const moe_attn_rows* q,
                           const moe_attn_rows* gate_or_null, float scale, void* o, void* ws, size_t ws_bytes,
                           moe_stream stream);

/* Causal attention of the last tokens of every sequence (a prompt, the rest of
 * a prompt over cached tokens, drafted tokens), n_tokens (up to 2^20) in all:
 * q, gate rows [n_tokens], o [n_tokens][q_heads][head_dim] (16-byte aligned). */
moe_status moe_attn_prefill(const moe_attn_desc* desc, const moe_kv_cache* cache, const int32_t* seq_off,
                            int32_t n_tokens, const moe_attn_rows* q, const moe_attn_rows* gate_or_null, float scale,
                            void* o, void* ws, size_t ws_bytes, moe_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_AMD_MOE_ATTN_H */
