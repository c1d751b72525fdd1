/*
 * moe_layer.h -- what stands around the experts' block of moe_experts.h: the
 * router with its gradient, and a whole mixture-of-experts layer for a few
 * tokens (router, experts, combine).  Part of the C ABI of libmoe_shuffle.so,
 * next to moe_shuffle.h, whose conventions hold here too: device pointers are
 * caller-owned, nothing is allocated, calls are asynchronous on `stream`,
 * every function returns a status code of moe_shuffle.h, and a failing call
 * writes no output.  dims are those of moe_shuffle.h; the calls here do not
 * look at num_ranks beyond its check.
 *
 * The routing rule, for a row x of H elements (bf16) and the router's weights
 * w_router [E][H] (bf16):
 *
 *   l_e = x . w_router[e]                              the logits
 *   s_e = exp(l_e - max l) / sum exp(l - max l)        scores (SOFTMAX), or
 *   s_e = 1 / (1 + exp(-l_e))                          (SIGMOID)
 *   key_e = l_e, or s_e + bias[e] where the rule has a bias (SIGMOID only)
 *   topk_idx    the k experts of the largest keys, largest first; of equal
 *               keys the lowest index first; a NaN counts as minus infinity
 *   topk_w[j] = scale s_j, or scale s_j / (sum over the k of s + 1e-20) where
 *               the rule normalizes                    the gates, fp32
 *
 * The choice of experts and their order are those of logits summed in 64 bits
 * (of exact products, in one order of additions that goes by H alone), whatever
 * the number of rows and whichever call routes them: a token is routed alike in
 * a long prompt, alone, and by moe_layer_forward.  Sums in 32 bits would swap
 * experts whose keys nearly tie, and another sum order would swap others.
 *
 * No output may overlap an input, another output or the workspace
 * (MOE_SHUFFLE_E_INVALID_ARG), but for `residual` and `grad_x_in`, which may be
 * the output that they are added to.  Row and weight pointers are 16-byte
 * aligned, the workspace 256, everything else 4 bytes.
 */
#ifndef MOE_LAYER_H
#define MOE_LAYER_H

#include "moe_experts.h"
#include "moe_shuffle.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Scores of a routing rule. */
enum {
    MOE_ROUTER_SOFTMAX = 0,
    MOE_ROUTER_SIGMOID = 1
};

typedef struct {
    int32_t scoring;   /* MOE_ROUTER_* */
    int32_t normalize; /* nonzero: the gates of a token sum to scale */
    float scale;       /* finite */
    int32_t reserved;  /* 0 */
    const float* bias; /* device fp32 [E], or NULL; with MOE_ROUTER_SIGMOID only */
} moe_router_rule;

/* Bytes of device workspace of the router's calls with these dims: of the
 * forward call, or, with `backward` nonzero, of both.  Scratch, 256-byte
 * aligned: nothing in it outlives a call, and calls that may overlap in time
 * (other streams, other captured graphs) need one each. */
int moe_router_workspace_size(const moe_shuffle_dims* dims, int32_t backward, size_t* bytes);

/*
 * Routes T rows.
 *   x         device bf16 [T, H];  w_router  device bf16 [E, H]
 *   topk_idx  device int32 [T, k], as moe_shuffle_plan takes it
 *   topk_w    device fp32 [T, k], as moe_shuffle_combine takes it
 *   logits    device fp32 [T, E], for the backward call; may be NULL
 * A logit is an fp32 sum in an order that the dims choose.  Limits: H < 2^20,
 * T * E and T * H below 2^40, and for the backward call T below 2^30.
 */
int moe_router_forward(const moe_shuffle_dims* dims, const moe_router_rule* rule, const void* x, const void* w_router,
                       int32_t* topk_idx, float* topk_w, float* logits, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * The router's backward pass, from the gates' gradients (grad_w of
 * moe_shuffle_combine_backward) to those of rows and weights; the choice of
 * experts has no gradient.  With g = scale grad_topk_w, and D the sum of the
 * chosen scores where the rule normalizes:
 *
 *   ds_j = g_j, or (g_j - sum_i g_i s_i / D) / D       for the chosen
 *   dl_e = ds_e s_e (1 - s_e)                          SIGMOID, 0 elsewhere
 *   dl_e = s_e (ds_e - sum_i ds_i s_i)                 SOFTMAX, ds 0 elsewhere
 *   dl  += grad_logits, where given (of a loss on the logits themselves)
 *   grad_x        = bf16(grad_x_in + dl w_router)                [T, H]
 *   grad_w_router = bf16(dl^T x)                                 [E, H]
 *
 * dl enters the matrix products, whose operands are bf16, as the sum of two
 * bf16 numbers: 16 bits of it count.  Sums are held in fp32.
 *   logits, topk_idx  as the forward call wrote them (bad ids: no result is
 *                     promised, nothing out of bounds is touched)
 *   grad_logits, grad_x_in  may be NULL; grad_x_in may be grad_x
 *   grad_x, grad_w_router   each may be NULL (it is not computed); w_router is
 *                     read for grad_x only and x for grad_w_router only, each
 *                     may be NULL where it is not read
 * With T = 0 grad_w_router is zero.
 */
int moe_router_backward(const moe_shuffle_dims* dims, const moe_router_rule* rule, const float* grad_topk_w,
                        const float* logits, const int32_t* topk_idx, const void* x, const void* w_router,
                        const float* grad_logits, const void* grad_x_in, void* grad_x, void* grad_w_router,
                        void* workspace, size_t workspace_bytes, void* stream);

/* The most tokens, and pairs of a token and an expert, of a layer's call. */
#define MOE_LAYER_MAX_TOKENS 64
#define MOE_LAYER_MAX_PAIRS 512

/* Bytes of device workspace of the layer's calls, scratch as above. */
int moe_layer_workspace_size(const moe_shuffle_dims* dims, int32_t inter, size_t* bytes);

/*
 * A whole layer for T <= 64 tokens, T * k <= 512 (else
 * MOE_SHUFFLE_E_OVERFLOW): routes x by the rule and computes
 *
 *   out[t] = bf16(residual[t] + sum_j topk_w[t][j] y_(topk_idx[t][j])(x[t]))
 *
 * with the experts' block y of moe_experts.h, its activations and its weights;
 * y is held in fp32 and summed in the order of j.
 *   residual  device bf16 [T, H], may be NULL, may be out
 *   out       device bf16 [T, H]
 *   topk_idx, topk_w  as of moe_router_forward; each may be NULL
 * Weights of experts that no token chose are not read.  A token's result does
 * not depend on the other tokens with the same dims.  Limits on H and inter
 * as in moe_experts.h.
 */
int moe_layer_forward(const moe_shuffle_dims* dims, const moe_router_rule* rule, const void* x, const void* w_router,
                      const void* w_gate_up, const void* w_down, int32_t inter, int32_t act, const void* residual,
                      void* out, int32_t* topk_idx, float* topk_w, void* workspace, size_t workspace_bytes,
                      void* stream);

/* The same with the 4-bit weights of moe_experts_ffn_w4_forward; the router's stay bf16. */
int moe_layer_w4_forward(const moe_shuffle_dims* dims, const moe_router_rule* rule, const void* x,
                         const void* w_router, const void* q_gate_up, const void* s_gate_up, const void* q_down,
                         const void* s_down, int32_t inter, int32_t group, int32_t act, const void* residual, void* out,
                         int32_t* topk_idx, float* topk_w, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYER_H */
