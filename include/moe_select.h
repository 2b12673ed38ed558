/*
 * moe_select.h - choosing K of E experts from router logits with scored,
 * biased and group-limited routing (beside moe_route's softmax top-K).
 *
 * Per token, for logits z[0..E):
 *
 *   live_e  = z_e is neither -inf nor NaN (an expert that is off is never chosen)
 *   score_e = 1 / (1 + exp(-z_e))                       MOE_SCORE_SIGMOID
 *           = exp(z_e - max z) / sum_live exp(z - max z)  MOE_SCORE_SOFTMAX
 *             (with an infinite maximum: the limit, equal shares of the
 *             experts at it); 0 for an expert that is off
 *   key_e   = score_e + bias_e      (bias: balance bias, enters the choice only;
 *             an expert whose key is -inf or NaN is off too)
 *   with top_groups < n_group: the E experts form n_group groups of
 *     E/n_group neighbours; a group's rank is the sum of its group_top
 *     largest live keys (-inf when none is live); only the experts of the
 *     top_groups groups of largest rank take part (ties: the lower group)
 *   S       = the K live experts of largest key (ties: the lower index), in
 *             that order; ranks without an expert get index -1 and weight 0
 *   w_k     = scale * score_{S_k}                        renorm = 0
 *           = scale * score_{S_k} / sum_j score_{S_j}    renorm = 1 (0 when the sum is 0)
 *
 * The order is that of the keys computed in 64 bits, so two experts come in
 * their true order however near their keys lie; weights are rounded to fp32
 * once.  moe_expert_ffn takes topk_idx / topk_w as they are (it skips index
 * -1).  The conventions of moe.h hold (caller-owned device buffers, work on
 * the given stream only, negative status and moe_last_error on refusal,
 * n_tokens == 0 a no-op); the results do not depend on the batch.
 */
#ifndef MOE_AMD_MOE_SELECT_H
#define MOE_AMD_MOE_SELECT_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_SCORE_SOFTMAX = 1, MOE_SCORE_SIGMOID = 2 };

/* n_experts E:  1..1024
 * top_k K:      1..min(E, 64)
 * score:        MOE_SCORE_*
 * n_group:      1..64, dividing E (0 is read as 1)
 * top_groups:   1..n_group with top_groups * E / n_group >= K (0 is read as n_group)
 * group_top:    1 or 2 (0 is read as 1); above the group's size it is that size
 * renorm:       0 or 1
 * scale:        finite */
typedef struct {
  int32_t n_experts, top_k, score, n_group, top_groups, group_top, renorm;
  float scale;
} moe_select_desc;

/* Choice from given logits.  logits: device fp32, row t at logits + t *
 * logits_stride (elements; >= E, >= E + 1 with shared_gate), as moe_route
 * writes them with logits_stride E + 1.  n_tokens up to 2^26 - 4.  bias: device fp32 [E] or NULL.
 * Outputs (device): topk_idx [T][K] int32, topk_w [T][K] fp32,
 * shared_gate_or_null [T] fp32 = sigmoid of column E of the logits. */
moe_status moe_select(const moe_select_desc* desc, const float* logits, int64_t logits_stride,
                      const float* bias_or_null, int32_t n_tokens, int32_t* topk_idx, float* topk_w,
                      float* shared_gate_or_null, moe_stream stream);

/* moe_route with this choice: router GEMV (logits without bias), then the
 * choice above with router_bias as the balance bias.  sel must agree with
 * desc in n_experts and top_k.  n_tokens as in moe_select, workspace and the
 * other arguments as in moe_route. */
moe_status moe_route_scored(const moe_layer_desc* desc, const moe_select_desc* sel, const moe_layer_weights* w,
                            const void* x, int32_t n_tokens, int32_t* topk_idx, float* topk_w, float* shared_gate,
                            float* logits_or_null, void* ws, size_t ws_bytes, moe_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_AMD_MOE_SELECT_H */
