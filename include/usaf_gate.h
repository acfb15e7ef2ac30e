/*
 * usaf_gate.h - C ABI of routing rules beyond usaf_route_topk's softmax top-k: scores by softmax or
 * sigmoid, a bias that balances the experts without entering the weights, experts taken from the best
 * groups only, weights renormalised and scaled; the gradient of such a rule, the bias's update, and the
 * experts' backward without the softmax router gradient that usaf_moe_bwd_sparse forms.
 *
 * The conventions of usaf.h hold: device pointers owned by the caller unless a comment says "host",
 * dense row-major tensors, no allocation, every call only enqueues on `stream`, host checks run before
 * anything is enqueued, conditions that only the device can see are OR-ed into *dev_status (which may
 * be NULL), no kernel traps. The USAF pages name no routing rule; these definitions are this library's.
 */
#ifndef USAF_GATE_H
#define USAF_GATE_H

#include "usaf.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { USAF_GATE_SOFTMAX = 0, USAF_GATE_SIGMOID = 1 } usaf_gate_score;

/* A routing rule (host). */
typedef struct {
  int32_t score;      /* usaf_gate_score */
  int32_t n_group;    /* groups of E / n_group consecutive experts; 1: none */
  int32_t topk_group; /* groups whose experts a token may take */
  int32_t group_top;  /* a group's score is the sum of its 1 or 2 largest choice scores */
  int32_t renorm;     /* 1: the weights of a token are divided by their sum */
  float scale;        /* weights are multiplied by it */
} usaf_gate;

/* ---------------------------------------------------------------------------------------------
 * usaf_gate_topk - router logits, experts and weights by the rule `gate`, token permutation.
 *   s[t,e] = softmax over e of logits[t,:], or 1 / (1 + exp(-logits[t,e]))
 *   c[t,e] = s[t,e] + bias[e]; -inf where the logit is -inf or NaN (an expert the token cannot take;
 *            softmax leaves it out)
 * With n_group > 1 a group's score is the sum of the group_top largest c of its experts (of those the
 * token can take, -inf if there is none); the topk_group groups with the largest scores are kept, ties
 * to the lower group, and c = -inf for the experts of the others. Per token the k experts with the
 * largest c are taken, in descending order, ties to the lower expert index. Order and choice are those
 * of c formed in 64 bits from the fp32 logits and bias (without a bias: of the logits), so they do not
 * depend on how fp32 scores round. Experts taken with c = -inf (fewer than k are left: the
 * lowest indices follow) have weight 0; the weights of the others are
 *   w_j = scale * s[t,e_j], divided by the sum of these s where renorm = 1 (the ratio is kept where the
 *         scores themselves are below the smallest fp32 numbers).
 *   gate       host
 *   x, x_dtype, w_router   as for usaf_route_topk; ignored when logits_in != NULL
 *   logits_in  [T,E] fp32 or NULL, row t at logits_in + t * ld_logits (ld_logits >= E)
 *   logits_out [T,E] fp32 or NULL: where computed logits are written
 *   bias       [E] fp32 or NULL (zero)
 *   rt         routing tables as usaf_route_topk writes them (all seven arrays required); topk_idx is
 *              in descending order of c
 *   dev_status gets USAF_DEV_NONFINITE for a NaN logit or bias, or a softmax logit of +inf (the
 *              token's weights are then NaN); USAF_DEV_TIMEOUT as for usaf_route_topk
 * The workspace must be 16-byte aligned (INVALID_ARG otherwise).
 * Limits: those of usaf_route_topk; 1 <= n_group <= 32, E % n_group == 0,
 * 1 <= topk_group <= n_group, k <= topk_group * E / n_group; scale finite and not 0.
 * Errors: INVALID_ARG, WORKSPACE, CUDA.
 * ------------------------------------------------------------------------------------------- */
size_t usaf_gate_topk_workspace_size(const usaf_moe_shape* shape);
usaf_status usaf_gate_topk(const usaf_moe_shape* shape, const usaf_gate* gate, const void* x,
                           usaf_dtype x_dtype, const float* w_router, const float* logits_in,
                           int64_t ld_logits, float* logits_out, const float* bias,
                           const usaf_routing* rt, uint32_t* dev_status, void* ws,
                           size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------------------------
 * usaf_gate_bwd - the gradient of the weights with respect to the logits, dw = dL/dw per slot (dw_slot
 * of usaf_moe_bwd_experts). The choice of experts, and slots with weight 0, are constants.
 *   u = sum_i w_i dw_i / scale where renorm = 1, else 0
 *   sigmoid:                dlogit[t,e_j] = w_j (dw_j - u) (1 - s[t,e_j])
 *   softmax, renorm = 1:    dlogit[t,e_j] = w_j (dw_j - u)
 *   softmax, renorm = 0:    dlogit[t,e]   = s[t,e] (scale dw_j [e = e_j] - sum_i w_i dw_i), every e
 * and 0 elsewhere.
 *   logits     [T,E] fp32, rows ld_logits apart; NULL will do for softmax with renorm = 1
 *   topk_idx, topk_w [T*k] as usaf_gate_topk wrote them;  dw [T*k] fp32
 *   dlogit     [T,E] fp32 out, rows ld_dlogit apart; accumulate = 1 adds to it. It may be the logits
 *              themselves (same pointer and stride) when accumulate = 0
 *   dev_status gets USAF_DEV_NONFINITE if a formed gradient is NaN/Inf, USAF_DEV_BAD_INDEX if an expert
 *              index is out of range (such slots are left out)
 * Limits: T >= 1, 1 <= k <= min(E, 32), E <= 1024, T*k < 2^31 - 65536. Errors: INVALID_ARG, CUDA.
 * ------------------------------------------------------------------------------------------- */
usaf_status usaf_gate_bwd(int64_t T, int64_t E, int64_t k, const usaf_gate* gate,
                          const float* logits, int64_t ld_logits, const int32_t* topk_idx,
                          const float* topk_w, const float* dw, float* dlogit, int64_t ld_dlogit,
                          int accumulate, uint32_t* dev_status, void* stream);

/* ---------------------------------------------------------------------------------------------
 * usaf_gate_balance - the step of the balancing bias: with c[e] = sum of count[:,e],
 *   bias[e] += rate * sign(mean(c) - c[e])
 * (experts that got less than their share become easier to choose). Counts are compared exactly.
 *   count [n,E] int32 (expert_count of a step's micro-batches, which has every slot; or the auxiliary
 *         losses' counts per group, which leave out the tokens that a mask does);  bias [E] fp32, updated
 *   skip_if_nonfinite  1: nothing moves if a bit of USAF_DEV_SKIP_MASK is set in *dev_status when the call
 *         runs, as with a step's other updates; 0: no check
 * Limits: 1 <= E <= 1024, 1 <= n <= 2^20; rate finite. Errors: INVALID_ARG, CUDA.
 * ------------------------------------------------------------------------------------------- */
usaf_status usaf_gate_balance(int64_t E, const int32_t* count, int64_t n, double rate, float* bias,
                              int skip_if_nonfinite, const uint32_t* dev_status, void* stream);

/* ---------------------------------------------------------------------------------------------
 * usaf_moe_bwd_experts - usaf_moe_bwd_sparse_planned without the router: g_act and dw_slot as there, dx
 * the experts' part alone, for weights that another rule than usaf_route_topk's formed. dw_slot
 * [T*k] is required; usaf_gate_bwd and usaf_router_grad (usaf_train.h) turn it into the router's
 * gradient and its part of dx.
 * Workspace: usaf_moe_bwd_workspace_size(shape, dtype, K). usaf_moe_wgrad_dense may follow.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA.
 * ------------------------------------------------------------------------------------------- */
usaf_status usaf_moe_bwd_experts(const usaf_moe_shape* shape, usaf_dtype dtype,
                                 const void* w_gate_up, const void* w_down, const usaf_routing* rt,
                                 const void* x_perm_save, const void* h_save, const void* wa_save,
                                 const void* dy, const int64_t* act_idx, int64_t K, float* g_act,
                                 void* dx, float* dw_slot, int accumulate, const void* plan,
                                 int64_t n_dense, uint32_t* dev_status, void* ws, size_t ws_bytes,
                                 void* stream);

#ifdef __cplusplus
}
#endif

#endif /* USAF_GATE_H */
