/*
 * moe_experts.h -- what the experts compute between dispatch and combine:
 * the gated feed-forward block on expert-major rows, its backward pass,
 * 8-bit activation checkpoints for that backward pass, and the same block
 * with 4-bit weights.  Part of the C ABI of libmoe_shuffle.so, next to
 * moe_shuffle.h, whose conventions hold here too: device pointers are
 * caller-owned, nothing is allocated, calls are asynchronous on `stream`,
 * every function returns a status code of moe_shuffle.h, and a failing call
 * writes no output.
 *
 * The rows q of expert e are [expert_offset[e], expert_offset[e+1]) of the
 * plan, known on the device only; P = T * k rows in all, of H elements each
 * (bf16).  I (`inter`) is the width between the two projections.  For each
 * expert, with its own weights:
 *
 *   g = x Wg^T, u = x Wu^T     the two projections          [I] each
 *   h = act(g) * u             fp32, rounded once to bf16   [I]
 *   y = h Wd^T                 rounded once to bf16         [H]
 *
 *   act(g) = g * sigmoid(a(g)),  a(g) = g                        (SiLU)
 *                                a(g) = 2 sqrt(2/pi) (g + 0.044715 g^3)
 *                                                 (GELU, its tanh form)
 *
 * Weights are bf16 and row-major, experts one after another:
 *   w_gate_up [E][2I][H]  rows [0, I) of an expert are Wg, [I, 2I) are Wu
 *   w_down    [E][H][I]   Wd
 *
 * Every sum is held in fp32 and rounded once.  Results depend on the inputs
 * alone: no atomics.  With the same dims and inter, a row's result depends on
 * that row and its expert's weights only, wherever the row lies and whatever
 * the other rows are.  The dims choose the kernel's form, and with it the order
 * in which a sum's terms are added: another number of tokens may round a row's
 * result differently.  A sigmoid below 2^-126 may be taken as 0.
 *
 * On a plan with bad top-k ids every call writes nothing, as the calls of
 * moe_shuffle.h do.  With T = 0 forward calls write nothing and return
 * MOE_SHUFFLE_OK; the backward call writes zero weight gradients.
 *
 * No output may overlap an input, another output, the workspace or the plan's
 * workspace (MOE_SHUFFLE_E_INVALID_ARG).
 *
 * Limits: I > 0, I % 8 == 0, H and I below 2^20, and all row and weight
 * pointers 16-byte aligned.  With Q = P + 1024, Q * ceil(I / 32) and
 * E * ceil(2I / 64) * ceil(H / 64) and Q * ceil(2 max(H, I) / 64) below 2^31
 * (MOE_SHUFFLE_E_OVERFLOW).
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_shuffle.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of the gate. */
enum {
    MOE_EXPERTS_ACT_SILU = 0,
    MOE_EXPERTS_ACT_GELU_TANH = 1
};

/* Elements along a row that share one scale in an 8-bit checkpoint. */
#define MOE_EXPERTS_GROUP8 32

/* Bytes of device workspace that the calls below need with these dims and
 * this `inter`: those of the forward calls (bf16 and 4-bit weights), or, with
 * `backward` nonzero, of the backward call too.  The workspace is 256-byte
 * aligned scratch: nothing in it outlives a call, and calls that may overlap
 * in time (other streams, other captured graphs) need one each. */
int moe_experts_ffn_workspace_size(const moe_shuffle_dims* dims, int32_t inter, int32_t backward, size_t* bytes);

/*
 * The block's forward pass, ye[q] = y(xe[q]) for every row.
 *   xe         device bf16 [P, H], expert-major as dispatch leaves it
 *   w_gate_up  device bf16 [E, 2I, H];  w_down  device bf16 [E, H, I]
 *   act        MOE_EXPERTS_ACT_*
 *   ye         device bf16 [P, H]
 *   saved, saved_scale  what the backward pass needs of the pre-activations:
 *     both NULL               nothing is kept (inference)
 *     saved alone             bf16 [P, 2I]: g, then u, each rounded to bf16
 *     both                    8-bit checkpoints: saved int8 [P, 2I],
 *                             saved_scale bf16 [P, 2, ceil(I / 32)], as
 *                             moe_experts_pack8 makes them of the fp32 g and
 *                             u (groups never span g and u)
 *   workspace  moe_experts_ffn_workspace_size(dims, inter, 0) bytes
 */
int moe_experts_ffn_forward(moe_shuffle_plan_t plan, const void* xe, const void* w_gate_up, const void* w_down,
                            int32_t inter, int32_t act, void* ye, void* saved, void* saved_scale, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * The block's backward pass from what forward saved (g and u below are the
 * values that `saved` holds):
 *   dh = grad_ye Wd,  h = act(g) u
 *   dg = bf16(dh u act'(g)),  du = bf16(dh act(g))
 *   grad_xe        = bf16(dg Wg + du Wu)                        [P, H]
 *   grad_w_gate_up = bf16([dg du]^T xe), expert by expert       [E, 2I, H]
 *   grad_w_down    = bf16(grad_ye^T bf16(h)), expert by expert  [E, H, I]
 * Gradients are written, not added; an expert with no rows gets zeros.
 * dg, du and h are rounded to bf16 because they are operands of bf16
 * matrix products, as h is in the forward pass.
 *   grad_xe may be NULL (it is not computed); so may grad_w_gate_up and
 *   grad_w_down, each (frozen weights).  xe is read for grad_w_gate_up only
 *   and w_gate_up for grad_xe only; each may be NULL where it is not read.
 *   saved, saved_scale  as forward wrote them
 *   workspace  moe_experts_ffn_workspace_size(dims, inter, 1) bytes
 */
int moe_experts_ffn_backward(moe_shuffle_plan_t plan, const void* grad_ye, const void* xe, const void* w_gate_up,
                             const void* w_down, int32_t inter, int32_t act, const void* saved,
                             const void* saved_scale, void* grad_xe, void* grad_w_gate_up, void* grad_w_down,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * The forward pass with 4-bit weights, for steps of few tokens, where the
 * bytes of the weights are the cost:
 *   w[n][c] = (q - 8) * scale[n][c / group],  q in 0 .. 15
 *   q_gate_up  device uint8 [E, 2I, H / 2], two columns a byte, the even
 *              column in the low four bits;   s_gate_up bf16 [E, 2I, H / group]
 *   q_down     device uint8 [E, H, I / 2];    s_down    bf16 [E, H, I / group]
 *   group      32, 64 or 128; H and I multiples of it (MOE_SHUFFLE_E_ALIGN)
 * A group's sum is sum q x - 8 sum x in fp32, scaled in fp32: no weight is
 * rounded, and what is lost is the fp32 rounding of 2 * group terms of up to
 * 15 |x|, also where q is 8.  An infinite x gives NaN, and so may finite ones
 * whose magnitudes in a group sum to 2^128 / 15 (2.2e37) or more; the same
 * goes for h in the down projection.  Any number of rows is computed; with
 * hundreds for an expert, bf16 weights are the faster form.  Other arguments
 * as for moe_experts_ffn_forward; all pointers 16-byte aligned.
 */
int moe_experts_ffn_w4_forward(moe_shuffle_plan_t plan, const void* xe, const void* q_gate_up, const void* s_gate_up,
                               const void* q_down, const void* s_down, int32_t inter, int32_t group, int32_t act,
                               void* ye, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Makes 4-bit weights of bf16 ones, row by row (rows: E * 2I or E * H):
 *   scale = bf16_rne(max |w| of the group / 7), at least 2^-126
 *   q     = min(max(rne(w * fp32(1 / scale)), -8), 7) + 8
 * A group that holds a NaN or an infinity gets scale NaN and q 8.
 *   w      device bf16 [rows, cols], cols % group == 0
 *   q      device uint8 [rows, cols / 2];  scale  device bf16 [rows, cols / group]
 */
int moe_experts_w4_quantize(const void* w, int64_t rows, int32_t cols, int32_t group, void* q, void* scale,
                            void* stream);

/*
 * 8-bit activation checkpoints of rows:
 *   step  = max(max |x| of the group / 127, 2^-126), rounded up to bf16
 *   q     = rne(x * fp32(1 / step)), in -127 .. 127
 *   x'    = q * step
 * A group is 32 elements along the row (the last may be shorter).  A group
 * that holds a NaN or an infinity gets step NaN and q 0: all of it comes
 * back as NaN.
 *   x      device bf16 [rows, cols], cols % 8 == 0
 *   q      device int8 [rows, cols];  scale  device bf16 [rows, ceil(cols / 32)]
 * unpack8 writes x' rounded to bf16 (one past bf16's range to its largest
 * finite value).  rows may be 0.
 */
int moe_experts_pack8(const void* x, int64_t rows, int32_t cols, void* q, void* scale, void* stream);
int moe_experts_unpack8(const void* q, const void* scale, int64_t rows, int32_t cols, void* x, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
