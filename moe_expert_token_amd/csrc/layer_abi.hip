// layer_abi.hip -- the extern "C" boundary of the router and of the layer for few tokens: argument checks and
// workspace sizes.
#include <hip/hip_runtime.h>

#include "checks.h"
#include "layer.h"

namespace {

using ms::Span;
using ms::misaligned;
using ms::overlaps;
using ms::status_of;

constexpr int kMaxWidth = 1 << 20;  // H and I below this: offsets inside a tile stay below 2^31

int check_rule(const moe_router_rule* r, ms::Rule* out)
{
    if (!r || r->reserved != 0) return MOE_SHUFFLE_E_INVALID_ARG;
    if (r->scoring != MOE_ROUTER_SOFTMAX && r->scoring != MOE_ROUTER_SIGMOID) return MOE_SHUFFLE_E_INVALID_ARG;
    if (!(r->scale >= -3.40282347e38f && r->scale <= 3.40282347e38f)) return MOE_SHUFFLE_E_INVALID_ARG;
    if (r->bias && r->scoring != MOE_ROUTER_SIGMOID) return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(r->bias, 4)) return MOE_SHUFFLE_E_ALIGN;
    *out = ms::Rule{r->scoring == MOE_ROUTER_SIGMOID, r->normalize != 0, r->scale, r->bias};
    return MOE_SHUFFLE_OK;
}

int check_layer(const moe_shuffle_dims* d, int32_t inter)
{
    const int rc = ms::check_dims(d);
    if (rc) return rc;
    if (inter <= 0) return MOE_SHUFFLE_E_INVALID_ARG;
    if (inter % 8 != 0) return MOE_SHUFFLE_E_ALIGN;
    if (inter >= kMaxWidth || d->hidden >= kMaxWidth) return MOE_SHUFFLE_E_OVERFLOW;
    if (d->num_tokens > ms::kLayerTokens || d->num_tokens * d->top_k > ms::kLayerPairs) return MOE_SHUFFLE_E_OVERFLOW;
    return MOE_SHUFFLE_OK;
}

ms::LayerShape layer_shape(const moe_shuffle_dims& d, int32_t inter)
{
    ms::LayerShape S{};
    S.T = d.num_tokens;
    S.H = d.hidden;
    S.E = d.num_experts;
    S.k = d.top_k;
    S.I = inter;
    S.P = S.T * S.k;
    return S;
}

// What both weights' calls share; the weights' sizes come with them.
int layer(const moe_shuffle_dims* dims, const moe_router_rule* rule, int32_t inter, int32_t act, ms::LayerCall C,
          size_t proj_bytes, size_t scale_bytes, void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_layer(dims, inter);
    ms::Rule q;
    if (!rc) rc = check_rule(rule, &q);
    if (rc) return rc;
    if (act != MOE_EXPERTS_ACT_SILU && act != MOE_EXPERTS_ACT_GELU_TANH) return MOE_SHUFFLE_E_INVALID_ARG;
    if (C.group && (dims->hidden % C.group || inter % C.group)) return MOE_SHUFFLE_E_ALIGN;
    ms::LayerShape S = layer_shape(*dims, inter);
    if (S.T == 0) return MOE_SHUFFLE_OK;
    if (!C.x || !C.w_router || !C.up || !C.down || !C.out || !workspace) return MOE_SHUFFLE_E_INVALID_ARG;
    if (C.group && (!C.up_scale || !C.down_scale)) return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(C.x, 16) || misaligned(C.w_router, 16) || misaligned(C.up, 16) || misaligned(C.up_scale, 16) ||
        misaligned(C.down, 16) || misaligned(C.down_scale, 16) || misaligned(C.residual, 16) || misaligned(C.out, 16) ||
        misaligned(C.topk_idx, 4) || misaligned(C.topk_w, 4) || misaligned(workspace, 256))
        return MOE_SHUFFLE_E_ALIGN;
    const size_t need = ms::layer_workspace(&S, (char*)workspace);
    if (workspace_bytes < need) return MOE_SHUFFLE_E_WORKSPACE;
    const size_t rows = (size_t)S.T * S.H * 2, pairs = (size_t)S.P * 4;
    const Span residual{C.residual == C.out ? nullptr : C.residual, rows};
    if (overlaps({{C.out, rows}, {C.topk_idx, pairs}, {C.topk_w, pairs}, {workspace, need}},
                 {{C.x, rows}, {C.w_router, (size_t)S.E * S.H * 2}, {C.up, 2 * proj_bytes}, {C.down, proj_bytes},
                  {C.up_scale, 2 * scale_bytes}, {C.down_scale, scale_bytes}, residual,
                  {q.bias, (size_t)S.E * 4}}))
        return MOE_SHUFFLE_E_INVALID_ARG;
    // 2 sqrt(2 / pi) = 1.5957691216
    S.c0 = act == MOE_EXPERTS_ACT_SILU ? 1.0f : 1.5957691216057308f;
    S.c1 = act == MOE_EXPERTS_ACT_SILU ? 0.0f : 1.5957691216057308f * 0.044715f;
    return status_of(ms::launch_layer(S, q, C, (hipStream_t)stream));
}

int check_router(const moe_shuffle_dims* d, bool backward)
{
    const int rc = ms::check_dims(d);
    if (rc) return rc;
    const int64_t T = d->num_tokens, lim = (int64_t)1 << 40;
    if (d->hidden >= kMaxWidth || T * d->num_experts >= lim || T * d->hidden >= lim || (backward && T >= 1 << 30))
        return MOE_SHUFFLE_E_OVERFLOW;
    return MOE_SHUFFLE_OK;
}

ms::RouterShape router_shape(const moe_shuffle_dims& d)
{
    return ms::RouterShape{d.num_tokens, d.hidden, d.num_experts, d.top_k};
}

int check_workspace(const void* workspace, size_t bytes, size_t need)
{
    if (!workspace) return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(workspace, 256)) return MOE_SHUFFLE_E_ALIGN;
    return bytes < need ? MOE_SHUFFLE_E_WORKSPACE : MOE_SHUFFLE_OK;
}

}  // namespace

extern "C" {

int moe_router_workspace_size(const moe_shuffle_dims* dims, int32_t backward, size_t* bytes)
{
    const int rc = check_router(dims, backward != 0);
    if (rc) return rc;
    if (!bytes) return MOE_SHUFFLE_E_INVALID_ARG;
    *bytes = ms::router_workspace(router_shape(*dims), backward != 0);
    return MOE_SHUFFLE_OK;
}

int moe_router_forward(const moe_shuffle_dims* dims, const moe_router_rule* rule, const void* x, const void* w_router,
                       int32_t* topk_idx, float* topk_w, float* logits, void* workspace, size_t workspace_bytes,
                       void* stream)
{
    int rc = check_router(dims, false);
    ms::Rule q;
    if (!rc) rc = check_rule(rule, &q);
    if (rc) return rc;
    const ms::RouterShape S = router_shape(*dims);
    if (S.T == 0) return MOE_SHUFFLE_OK;
    if (!x || !w_router || !topk_idx || !topk_w) return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(w_router, 16) || misaligned(topk_idx, 4) || misaligned(topk_w, 4) ||
        misaligned(logits, 4))
        return MOE_SHUFFLE_E_ALIGN;
    const size_t need = ms::router_workspace(S, false), pairs = (size_t)S.T * S.k * 4;
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc) return rc;
    if (overlaps({{topk_idx, pairs}, {topk_w, pairs}, {logits, (size_t)S.T * S.E * 4}, {workspace, need}},
                 {{x, (size_t)S.T * S.H * 2}, {w_router, (size_t)S.E * S.H * 2}, {q.bias, (size_t)S.E * 4}}))
        return MOE_SHUFFLE_E_INVALID_ARG;
    return status_of(ms::launch_router_forward(S, q, x, w_router, topk_idx, topk_w, logits, (char*)workspace,
                                               (hipStream_t)stream));
}

int moe_router_backward(const moe_shuffle_dims* dims, const moe_router_rule* rule, const float* grad_topk_w,
                        const float* logits, const int32_t* topk_idx, const void* x, const void* w_router,
                        const float* grad_logits, const void* grad_x_in, void* grad_x, void* grad_w_router,
                        void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_router(dims, true);
    ms::Rule q;
    if (!rc) rc = check_rule(rule, &q);
    if (rc) return rc;
    const ms::RouterShape S = router_shape(*dims);
    // with no rows only the (zero) weights' gradient is written, and nothing is read
    if (S.T > 0 && (!grad_topk_w || !logits || !topk_idx || (grad_x && !w_router) || (grad_w_router && !x)))
        return MOE_SHUFFLE_E_INVALID_ARG;
    if (grad_x_in && !grad_x) return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(w_router, 16) || misaligned(grad_x_in, 16) || misaligned(grad_x, 16) ||
        misaligned(grad_w_router, 16) || misaligned(grad_topk_w, 4) || misaligned(logits, 4) ||
        misaligned(topk_idx, 4) || misaligned(grad_logits, 4))
        return MOE_SHUFFLE_E_ALIGN;
    const size_t need = ms::router_workspace(S, true), pairs = (size_t)S.T * S.k * 4;
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc) return rc;
    const size_t rows = (size_t)S.T * S.H * 2, weights = (size_t)S.E * S.H * 2, table = (size_t)S.T * S.E * 4;
    if (overlaps({{grad_x, rows}, {grad_w_router, weights}, {workspace, need}},
                 {{x, rows}, {w_router, weights}, {grad_topk_w, pairs}, {logits, table}, {topk_idx, pairs},
                  {grad_logits, table}, {grad_x_in == grad_x ? nullptr : grad_x_in, rows}}))
        return MOE_SHUFFLE_E_INVALID_ARG;
    if (!grad_x && !grad_w_router) return MOE_SHUFFLE_OK;
    return status_of(ms::launch_router_backward(S, q, grad_topk_w, logits, topk_idx, x, w_router, grad_logits,
                                                grad_x_in, grad_x, grad_w_router, (char*)workspace,
                                                (hipStream_t)stream));
}

int moe_layer_workspace_size(const moe_shuffle_dims* dims, int32_t inter, size_t* bytes)
{
    const int rc = check_layer(dims, inter);
    if (rc) return rc;
    if (!bytes) return MOE_SHUFFLE_E_INVALID_ARG;
    ms::LayerShape S = layer_shape(*dims, inter);
    *bytes = ms::layer_workspace(&S, nullptr);
    return MOE_SHUFFLE_OK;
}

int moe_layer_forward(const moe_shuffle_dims* dims, const moe_router_rule* rule, const void* x, const void* w_router,
                      const void* w_gate_up, const void* w_down, int32_t inter, int32_t act, const void* residual,
                      void* out, int32_t* topk_idx, float* topk_w, void* workspace, size_t workspace_bytes,
                      void* stream)
{
    const size_t proj = dims && inter > 0 ? (size_t)dims->num_experts * inter * dims->hidden * 2 : 0;
    return layer(dims, rule, inter, act,
                 ms::LayerCall{x, w_router, w_gate_up, nullptr, w_down, nullptr, residual, out, topk_idx, topk_w, 0},
                 proj, 0, workspace, workspace_bytes, stream);
}

int moe_layer_w4_forward(const moe_shuffle_dims* dims, const moe_router_rule* rule, const void* x,
                         const void* w_router, const void* q_gate_up, const void* s_gate_up, const void* q_down,
                         const void* s_down, int32_t inter, int32_t group, int32_t act, const void* residual, void* out,
                         int32_t* topk_idx, float* topk_w, void* workspace, size_t workspace_bytes, void* stream)
{
    if (group != 32 && group != 64 && group != 128) return MOE_SHUFFLE_E_INVALID_ARG;
    const size_t proj = dims && inter > 0 ? (size_t)dims->num_experts * inter * dims->hidden / 2 : 0;
    return layer(dims, rule, inter, act,
                 ms::LayerCall{x, w_router, q_gate_up, s_gate_up, q_down, s_down, residual, out, topk_idx, topk_w, group},
                 proj, proj * 4 / group, workspace, workspace_bytes, stream);
}

}  // extern "C"
