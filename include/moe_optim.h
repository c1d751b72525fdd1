/*
 * moe_optim.h -- the optimizer's step on what the backward calls of
 * moe_experts.h and moe_layer.h give: AdamW over many tensors at once, with
 * its states in fp32 or in 8 bits.  Part of the C ABI of libmoe_shuffle.so,
 * next to moe_shuffle.h, whose conventions hold here too: device pointers are
 * caller-owned, nothing is allocated, calls are asynchronous on `stream`,
 * every function returns a status code of moe_shuffle.h, and a failing call
 * launches nothing.
 *
 * For every element, in fp32:
 *
 *   g' = grad_scale g
 *   m  = beta1 m + (1 - beta1) g'
 *   v  = beta2 v + (1 - beta2) g'^2
 *   p  = (1 - lr weight_decay) p
 *        - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 *
 * The constants (1 - beta, the powers, the root) are taken in 64 bits and
 * rounded once.  A bf16 parameter is rounded to nearest: a step of less than
 * 2^-9 of it is lost, so training over many steps wants fp32 parameters, with
 * `copy` for the bf16 weights that the products read.
 *
 * 8-bit states.  128 neighbouring elements of a tensor share two fp32 steps;
 * with the group's largest magnitudes top_m of m and top_s of s = sqrt(v):
 *
 *   m_scale = max(top_m * fp32(1 / 448), 2^-126),   m is e4m3(m * fp32(1 / m_scale))
 *   v_scale = max(top_s * fp32(1 / 8064), 2^-126),  s is an unsigned float of
 *             three exponent and five mantissa bits: code c > 0 stands for
 *             (32 + c % 32) 2^(c / 32) v_scale, code 0 for 0; the nearest
 *             code, the even one of two, and never 0 for s > 0
 *
 * so that what is read back is off by half a step of e4m3 (2^-4 of m, down
 * to 2^-10 of m_scale) and by 2^-6 of s.  s below v_scale * 33 comes back as
 * that, 1/244 of the group's largest: such an element takes smaller steps.
 * A second moment changes by a thousandth a step (beta2 = 0.999), which no
 * 8-bit scale could follow: that is why the steps are fp32, and the largest of
 * a group moves exactly.  A group in which m or s is not finite gets the
 * scale NaN: all of it reads back as NaN.  All-zero states (codes and
 * scales) are those of a first step.
 *
 * Limits: count >= 0, 0 <= n < 2^40 each, pointers 16-byte aligned (scales 4).
 * The tensors of a call must not
 * overlap each other; within one of them that is checked.
 */
#ifndef MOE_OPTIM_H
#define MOE_OPTIM_H

#include "moe_shuffle.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of parameters, gradients, states, and values of states. */
enum {
    MOE_ADAMW_F32 = 0,
    MOE_ADAMW_BF16 = 1, /* not for states */
    MOE_ADAMW_8BIT = 2  /* states only */
};

/* Elements that share the scales of 8-bit states. */
#define MOE_ADAMW_GROUP 128

/* One tensor of n elements; device pointers.  With n = 0 none is read. */
typedef struct {
    void* p;          /* parameters, read and written */
    void* copy;       /* NULL, or bf16: the new (fp32) parameters rounded to nearest */
    const void* g;    /* gradients */
    void* m;          /* first moments: fp32, or codes of one byte */
    void* v;          /* second moments: fp32, or codes of one byte of their roots */
    float* m_scale;   /* [ceil(n / 128)], 8-bit states only */
    float* v_scale;
    void* m_out;      /* the states' values, for moe_adamw_pack and _unpack only */
    void* v_out;
    int64_t n;
} moe_adamw_tensor;

typedef struct {
    int32_t param, grad, state; /* MOE_ADAMW_*, of every tensor of the call */
    int32_t reserved;           /* 0 */
    double lr, beta1, beta2, eps, weight_decay; /* betas in [0, 1), lr, eps and weight_decay >= 0, all finite */
    int64_t step;               /* 1 for the first */
    /* device scalars, each may be NULL; read when the kernels run, so that a captured graph follows them */
    const float* lr_device;      /* in place of lr */
    const int64_t* step_device;  /* in place of step; below 1 it counts as 1 */
    const float* grad_scale;     /* factor of every gradient, 1 where NULL (clipping by the global norm) */
} moe_adamw_params;

/*
 * The step, on all tensors: one launch for every 40 of them.
 *   tensors  host array of `count`, read during the call
 */
int moe_adamw_step(const moe_adamw_tensor* tensors, int32_t count, const moe_adamw_params* params, void* stream);

/*
 * 8-bit states of a tensor's fp32 m_out and v_out (loading a checkpoint), and
 * the values that 8-bit states hold into m_out and v_out, which are fp32 or
 * bf16 by `values` (writing one).  v_out holds v, not its root; a v below 0
 * counts as 0.  p, copy and g are not looked at.
 */
int moe_adamw_pack(const moe_adamw_tensor* tensors, int32_t count, void* stream);
int moe_adamw_unpack(const moe_adamw_tensor* tensors, int32_t count, int32_t values, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPTIM_H */
