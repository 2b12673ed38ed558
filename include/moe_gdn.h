/*
 * moe_gdn.h - Gated DeltaNet recurrence (the linear attention that runs
 * beside the MoE block): one token per sequence, or whole sequences.
 *
 * Three quarters of the layers of the models this library serves use Gated
 * DeltaNet linear attention with a fixed-size recurrent state instead of a
 * growing KV cache (page "Show HN: Run an 80B Qwen in 4.3 GB of RAM on a Mac
 * and a 35B on an iPhone", how-it-works list).  The pages give no formula;
 * this is the published gated delta rule (Yang, Kautz and Hatamizadeh,
 * "Gated Delta Networks: Improving Mamba2 with Delta Rule", ICLR 2025), one
 * decode token per sequence, per value head h with key head
 * hk = h / (v_heads / k_heads):
 *
 *   k^ = k[hk] / sqrt(|k[hk]|^2 + 1e-6)
 *   q^ = q_scale * q[hk] / sqrt(|q[hk]|^2 + 1e-6)
 *   alpha = exp(g[h]),   b = beta[h]
 *   S' = alpha S + b (v[h] - alpha S k^) k^T          (S: [d_v][d_k])
 *   o[h] = S' q^
 *
 * Buffers (device, caller-owned):
 *   q, k:   [B][k_heads][d_k]  act_dtype, 8-byte aligned
 *   v:      [B][v_heads][d_v]  act_dtype, 2-byte aligned
 *   g, beta:[B][v_heads]       fp32 (g <= 0 is the log of the decay)
 *   state:  [B][v_heads][d_v][d_k] fp32, 16-byte aligned, updated in place
 *   o:      [B][v_heads][d_v]  fp32
 * Products and sums are fp32 in a fixed order (bitwise repeatable); the
 * state stays fp32.  Only the given stream is used.
 */
#ifndef MOE_AMD_MOE_GDN_H
#define MOE_AMD_MOE_GDN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape of one Gated DeltaNet layer step.
 *   batch:      B in [0, 65535] (0 is a no-op)
 *   k_heads:    >= 1
 *   v_heads:    a multiple of k_heads, <= 1024
 *   head_k_dim: 128
 *   head_v_dim: a multiple of 16, 16..256
 *   act_dtype:  MOE_F16 or MOE_BF16 (q, k, v) */
typedef struct {
  int32_t batch, k_heads, v_heads, head_k_dim, head_v_dim, act_dtype;
} moe_gdn_desc;

/* One token of the recurrence for every sequence and value head.  MOE_ESHAPE
 * for unsupported sizes, MOE_EINVAL for NULL or misaligned pointers or a bad
 * act_dtype; nothing is enqueued then. */
moe_status moe_gdn_step(const moe_gdn_desc* desc, const void* q, const void* k, const void* v, const float* g,
                        const float* beta, float q_scale, float* state, float* o, moe_stream stream);

/* The same rule over whole sequences (prompts, or several drafted tokens):
 * the tokens of B sequences lie one after the other in q, k, v, g, beta and o
 * ([n_tokens][heads]... as above, token rows instead of sequence rows), and
 * sequence b owns tokens seq_off[b] .. seq_off[b+1] - 1 (device int32 [B+1],
 * non-decreasing, within [0, n_tokens]).  state [B][v_heads][d_v][d_k] holds
 * each sequence's state on entry and after its last token on exit; a sequence
 * without tokens keeps its state.  Rows of o outside every sequence are left
 * as they are.  Offsets outside the range are read as its nearest end, and an
 * end before its start as an empty sequence: no access leaves the buffers, but
 * where offsets decrease the results are not defined.
 *
 * desc->batch is B; q, k 16-byte aligned; n_tokens up to 2^30 and
 * n_tokens / 64 + B below 2^24.  The workspace (256-byte aligned,
 * moe_gdn_prefill_workspace_bytes) is only used while the call runs; above 24
 * tokens it holds 48 KB for each key head and 25 KB for each value head of
 * n_tokens / 64 + B blocks (8192 tokens of one sequence, 16 and 32 heads: 207 MB).
 *
 * State and sums are fp32; the results are those of the tokens taken one by one
 * up to fp32 rounding (in a block of 64 tokens, see below, also up to 2^-40 of
 * the block's largest value and of the state before it: what a block shrinks
 * further than that may become 0, for the tokens after it too), bitwise
 * repeatable, and a sequence's results do not depend on the other sequences.
 * Any g and beta work whose states stay in fp32's range (g = -inf clears the
 * state), but g <= 0 and beta in [0, 2] are expected: with more than 24 tokens,
 * a sequence and value head is taken in blocks of 64 tokens up to its first
 * block with another g or beta, and token by token, some 15 times slower, from
 * there on.  A non-finite k, v, beta or g makes that sequence's results unusable
 * from the start of its 64-token block on.  A row of q or k whose sum of squares
 * overflows fp32 counts as zero. */
moe_status moe_gdn_prefill_workspace_bytes(const moe_gdn_desc* desc, int32_t n_tokens, size_t* bytes);
moe_status moe_gdn_prefill(const moe_gdn_desc* desc, const int32_t* seq_off, int32_t n_tokens, const void* q,
                           const void* k, const void* v, const float* g, const float* beta, float q_scale,
                           float* state, float* o, void* ws, size_t ws_bytes, moe_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_AMD_MOE_GDN_H */
