/*
 * usaf_train.h - C ABI of what a train step of a USAF MoE layer may add to the calls of usaf.h:
 * auxiliary losses of the router with their gradients, the products of a dense router gradient,
 * and activations kept in 8 bits between the forward and the backward.
 *
 * The conventions of usaf.h hold: device pointers owned by the caller unless a comment says
 * "host", dense row-major tensors, no allocation (scratch comes from a workspace sized by the
 * *_workspace_size query, a host-only computation that returns 0 for sizes a call would refuse),
 * every call only enqueues on `stream`, host checks run before anything is enqueued, conditions
 * that only the device can see are OR-ed into *dev_status (which may be NULL), no kernel traps.
 * The USAF pages train the router in full ("The router is leverage") and do not mention these
 * losses or an activation format; the definitions below are this library's.
 */
#ifndef USAF_TRAIN_H
#define USAF_TRAIN_H

#include "usaf.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------------------------
 * usaf_router_aux_fwd - load-balance loss, z-loss and per-expert counts of a router's logits.
 * Tokens come in G groups of consecutive tokens (packed sequences), or in one. A token takes part
 * unless its mask is 0, it is in no group, or its logits are all -inf. With c[g,e] the slots of
 * group g's tokens that are routed to e, P[g,e] the sum of their softmax probabilities (over all E
 * logits), n[g] their number and n = sum_g n[g]:
 *   balance = E / (k n) sum_g 1/n[g] sum_e c[g,e] P[g,e]   (1 for a perfectly even router; each
 *             group's own E sum_e (c/(k n[g])) (P/n[g]), weighted by its tokens)
 *   z       = 1/n sum_t logsumexp_e(logits[t,e])^2
 *   loss    = { coef_balance balance + coef_z z, balance, z };  all 0 when n = 0
 *   logits       [T,E] fp32, row t at logits + t * ld_logits (ld_logits >= E); -inf entries are
 *                experts the token cannot take; masked tokens' are ignored
 *   topk_idx     [T*k] expert of each slot, as usaf_route_topk writes it
 *   token_mask   [T] bytes, 0 = the token does not take part; NULL: every token does
 *   group_offset [G+1] first token of each group, non-decreasing; tokens before the first or from
 *                the last offset on are in no group. NULL with G = 1: one group of all tokens
 *   count, prob_sum [G,E] out (int32 c, fp32 P);  n_tok [G] out (int32 n);  loss [3] out
 *   dev_status   gets USAF_DEV_NONFINITE if the loss is NaN/Inf (a NaN or +inf logit of a token
 *                that takes part makes it so), USAF_DEV_BAD_INDEX if an expert index or a group
 *                offset is out of range or the offsets decrease (such slots are not counted, such
 *                offsets are clamped)
 * A term whose coefficient is 0 is still reported in loss[1] / loss[2] and adds nothing to loss[0].
 * All sums have a fixed order: the same inputs give the same bits.
 * The workspace must be 16-byte aligned (INVALID_ARG otherwise).
 * Limits: T >= 1, 1 <= k <= min(E, 32), E <= 1024, 1 <= G <= 2^20, T*k < 2^31 - 65536.
 * Errors: INVALID_ARG, WORKSPACE, CUDA.
 * ------------------------------------------------------------------------------------------- */
size_t usaf_router_aux_workspace_size(int64_t T, int64_t E, int64_t k, int64_t G);
usaf_status usaf_router_aux_fwd(int64_t T, int64_t E, int64_t k, const float* logits,
                                int64_t ld_logits, const int32_t* topk_idx,
                                const uint8_t* token_mask, const int32_t* group_offset, int64_t G,
                                double coef_balance, double coef_z, int32_t* count,
                                float* prob_sum, int32_t* n_tok, float* loss,
                                uint32_t* dev_status, void* ws, size_t ws_bytes, void* stream);

/* usaf_router_aux_bwd - the gradient of loss[0] with respect to the logits (counts are constants):
 *   dlogit[t,e] = d_loss p[t,e] ( coef_balance E/(k n n[g]) (c[g,e] - sum_j p[t,j] c[g,j])
 *                                 + coef_z 2/n logsumexp(logits[t]) )
 * and 0 for tokens that take no part and where p = 0 (a logit of -inf), whatever d_loss is.
 *   count, n_tok  as usaf_router_aux_fwd wrote them, or summed over ranks (with one group) for the
 *                 gradient of a whole data-parallel batch's loss
 *   d_loss        [1] fp32 upstream gradient, or NULL for 1
 *   dlogit        [T,E] fp32 out, rows ld_dlogit apart; accumulate = 1 adds to it. It may be the
 *                 logits themselves (same pointer and stride) when accumulate = 0
 *   dev_status    gets USAF_DEV_NONFINITE if a produced gradient is NaN/Inf, USAF_DEV_BAD_INDEX
 *                 for group offsets as above
 * The other arguments, limits and errors as for the forward (no workspace). */
usaf_status usaf_router_aux_bwd(int64_t T, int64_t E, int64_t k, const float* logits,
                                int64_t ld_logits, const uint8_t* token_mask,
                                const int32_t* group_offset, int64_t G, double coef_balance,
                                double coef_z, const int32_t* count, const int32_t* n_tok,
                                const float* d_loss, float* dlogit, int64_t ld_dlogit,
                                int accumulate, uint32_t* dev_status, void* stream);

/* ---------------------------------------------------------------------------------------------
 * usaf_router_grad - the two products of a dense router gradient dlogit = dL/dlogits:
 *   g_router[e,h] = g_in[e,h]  + sum_t dlogit[t,e] x[t,h]
 *   dx[t,h]       = dx_in[t,h] + sum_e dlogit[t,e] w_router[e,h]
 * (usaf_moe_bwd_sparse forms them for the k selected experts of each token; an auxiliary loss
 * moves every logit.)
 *   dlogit    [T,E] fp32, rows ld_dlogit apart (ld_dlogit >= E)
 *   dtype     of x, dx_in and dx, [T,H]: USAF_BF16 (H % 64 == 0) on tcgen05 tensor cores, or
 *             USAF_F32 (any H) on CUDA cores
 *   x         needed for g_router;  w_router [E,H] fp32, needed for dx
 *   g_in      [E,H] fp32 or NULL (zero);  g_router [E,H] fp32 out, or NULL to skip; may be g_in
 *   dx_in     [T,H] or NULL (zero);  dx [T,H] out, or NULL to skip; may be dx_in
 *             Neither output may overlap any other input (dx = x is refused where g_router is
 *             asked for, whose product reads x).
 *   dev_status gets USAF_DEV_NONFINITE if a produced gradient is NaN/Inf (of bf16 layers an infinite
 *              dlogit or w_router gives NaN), USAF_DEV_TIMEOUT if a tensor-core kernel gave up a wait
 * Sums are fp32, their order is fixed. On tensor cores dlogit and w_router are carried exactly, as
 * three bf16 parts each; of dx's products of two parts those below 2^-24 of the whole are left out.
 * The workspace and, of bf16 layers, x, dx_in, dx and w_router must be 16-byte aligned (INVALID_ARG
 * otherwise).
 * Limits: T >= 1, 1 <= E <= 1024, H >= 1, T < 2^31 - 65536, E*H < 2^31.
 * Errors: INVALID_ARG, UNSUPPORTED (bf16 with H % 64 != 0; fp32 beyond 2^31 tiles of 64 x 64),
 * WORKSPACE, CUDA.
 * ------------------------------------------------------------------------------------------- */
size_t usaf_router_grad_workspace_size(int64_t T, int64_t E, int64_t H, usaf_dtype dtype);
usaf_status usaf_router_grad(int64_t T, int64_t E, int64_t H, usaf_dtype dtype,
                             const float* dlogit, int64_t ld_dlogit, const void* x,
                             const float* w_router, const float* g_in, float* g_router,
                             const void* dx_in, void* dx, uint32_t* dev_status, void* ws,
                             size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Activations in 8 bits. Between a layer's forward and its backward usaf.h keeps x_perm, h and wa
 * (H + 3I values of 2 or 4 bytes per routed row) and x. usaf_act8_save keeps x and h instead, in
 * 17/16 bytes a value; usaf_act8_restore turns them back into what the backward reads: x_perm is
 * x gathered, wa = w silu(gate) up again. A stack of layers then needs one x_perm, h and wa.
 * Format: blocks of USAF_ACT8_BLOCK consecutive values (of a token's features in x, the last block
 * of a token may be short; of a feature's permuted rows in h, where no block crosses experts,
 * because their rows start at multiples of 16). With amax the block's largest magnitude, e is the
 * least exponent with amax <= 127 * 2^e, at least -126 and at most 121; a code is v * 2^-e rounded
 * to nearest even (and to +-127), the exponent byte e + 127. A block of zeros has byte 0, a block
 * with a NaN or infinity byte 255 and codes 0; a value is code * 2^(byte - 127), 0 for byte 0 and
 * NaN for byte 255. Codes have 7 bits, so a value is exact in bf16.
 *   x_code [T,H] int8,       x_exp [T, ceil(H/16)]   uint8
 *   h_code [2I,R_cap] int8,  h_exp [2I, R_cap/16]    uint8   (rows past expert_offset[E] unused)
 * usaf_act8_save: x [T,H] and h [2I,R_cap] (as usaf_moe_fwd left them) of dtype, rt the routing
 *   of that forward. dev_status gets USAF_DEV_NONFINITE if a block holds a NaN or infinity.
 * usaf_act8_restore: x_out [T,H] (or NULL), x_perm [H,R_cap], h [2I,R_cap], wa [I,R_cap] out, of
 *   dtype, with the same routing (topk_w, expert_offset, perm_tok, perm_slot are read). Padding
 *   rows come out 0 (in h and wa unless their block is NaN); of the rows past expert_offset[E],
 *   x_perm's are 0 and those of h and wa may be left as they were, as after a forward.
 * All pointers of the store and the tensors, perm_tok and perm_slot must be 16-byte aligned.
 * Any T, H, E, k, I of a valid shape, both dtypes.
 * Errors: INVALID_ARG, UNSUPPORTED (a restore beyond 2^31 blocks of work), CUDA.
 * ------------------------------------------------------------------------------------------- */
#define USAF_ACT8_BLOCK 16
usaf_status usaf_act8_save(const usaf_moe_shape* shape, usaf_dtype dtype, const void* x,
                           const void* h, const usaf_routing* rt, int8_t* x_code, uint8_t* x_exp,
                           int8_t* h_code, uint8_t* h_exp, uint32_t* dev_status, void* stream);
usaf_status usaf_act8_restore(const usaf_moe_shape* shape, usaf_dtype dtype, const int8_t* x_code,
                              const uint8_t* x_exp, const int8_t* h_code, const uint8_t* h_exp,
                              const usaf_routing* rt, void* x_out, void* x_perm, void* h,
                              void* wa, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* USAF_TRAIN_H */
