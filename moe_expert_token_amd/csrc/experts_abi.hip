// experts_abi.hip -- the extern "C" boundary of the experts' block: argument
// checks, workspace layout and launches.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "experts.h"
#include "internal.h"

namespace {

constexpr int kTileRoom = 1024;
constexpr int kMaxWidth = 1 << 20;  // H and I below this: offsets inside a tile stay below 2^31

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Span {
    const void* p;
    size_t bytes;
};

// Whether any of `outs` overlaps another of them or any of `ins`.
bool overlaps(std::initializer_list<Span> outs, std::initializer_list<Span> ins)
{
    const auto hit = [](const Span& a, const Span& b) {
        if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
        const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
        return x < y + b.bytes && y < x + a.bytes;
    };
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (auto q = o + 1; q != outs.end(); ++q)
            if (hit(*o, *q)) return true;
        for (const Span& i : ins)
            if (hit(*o, i)) return true;
    }
    return false;
}

int check_inter(const moe_shuffle_dims& d, int32_t inter)
{
    if (inter <= 0) return MOE_SHUFFLE_E_INVALID_ARG;
    if (inter % 8 != 0) return MOE_SHUFFLE_E_ALIGN;
    if (inter >= kMaxWidth || d.hidden >= kMaxWidth) return MOE_SHUFFLE_E_OVERFLOW;
    // the kernels round row counts up to tiles, and count tiles and pieces of rows with int
    const int64_t P = (int64_t)d.num_tokens * d.top_k + kTileRoom, lim = (int64_t)1 << 31;
    const int64_t wide = d.hidden > inter ? d.hidden : inter;
    const int64_t up = (2 * (int64_t)inter + 63) / 64, hid = ((int64_t)d.hidden + 63) / 64;
    if (P * ((inter + 31) / 32) >= lim || P * ((2 * wide + 63) / 64) >= lim || d.num_experts * up * hid >= lim)
        return MOE_SHUFFLE_E_OVERFLOW;
    return MOE_SHUFFLE_OK;
}

// Checks what every call on a plan has, and fills the shape.
int expert_shape(moe_shuffle_plan_t plan, int32_t inter, int32_t act, ms::ExpertShape* S)
{
    if (!plan || !plan->ws) return MOE_SHUFFLE_E_INVALID_ARG;
    const int rc = check_inter(plan->dims, inter);
    if (rc) return rc;
    if (act != MOE_EXPERTS_ACT_SILU && act != MOE_EXPERTS_ACT_GELU_TANH) return MOE_SHUFFLE_E_INVALID_ARG;
    const ms::Layout& L = plan->L;
    S->P = L.T * L.k;
    S->H = L.H;
    S->I = inter;
    S->E = L.E;
    // 2 sqrt(2 / pi) = 1.5957691216
    S->c0 = act == MOE_EXPERTS_ACT_SILU ? 1.0f : 1.5957691216057308f;
    S->c1 = act == MOE_EXPERTS_ACT_SILU ? 0.0f : 1.5957691216057308f * 0.044715f;
    S->offset = (const int32_t*)(plan->ws + L.expert_offset);
    S->status = (const int32_t*)(plan->ws + L.status);
    return MOE_SHUFFLE_OK;
}

size_t hidden_bytes(const ms::ExpertShape& S) { return align256((size_t)S.P * S.I * 2); }

// The forward calls keep h in the workspace; the backward call h, [dg du] behind it.
size_t workspace_bytes_of(const ms::ExpertShape& S, bool backward)
{
    const size_t n = hidden_bytes(S) * (backward ? 3 : 1);
    return n ? n : 256;
}

int check_workspace(const ms::ExpertShape& S, bool backward, const void* workspace, size_t bytes)
{
    if (!workspace) return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(workspace, 256)) return MOE_SHUFFLE_E_ALIGN;
    return bytes < workspace_bytes_of(S, backward) ? MOE_SHUFFLE_E_WORKSPACE : MOE_SHUFFLE_OK;
}

// Bytes of what forward saves and of its scales.
size_t saved_bytes(const ms::ExpertShape& S, bool eight) { return (size_t)S.P * 2 * S.I * (eight ? 1 : 2); }
size_t scale_bytes(const ms::ExpertShape& S) { return (size_t)S.P * 2 * ((S.I + ms::kGroup8 - 1) / ms::kGroup8) * 2; }

// The plan's own workspace, which nothing may write.
Span plan_span(moe_shuffle_plan_t plan) { return Span{plan->ws, plan->L.total}; }

int status_of(hipError_t e) { return e == hipSuccess ? MOE_SHUFFLE_OK : ms::hip_fail(e); }

}  // namespace

extern "C" {

int moe_experts_ffn_workspace_size(const moe_shuffle_dims* dims, int32_t inter, int32_t backward, size_t* bytes)
{
    int rc = ms::check_dims(dims);
    if (!rc) rc = check_inter(*dims, inter);
    if (rc) return rc;
    if (!bytes) return MOE_SHUFFLE_E_INVALID_ARG;
    ms::ExpertShape S{};
    S.P = dims->num_tokens * dims->top_k;
    S.I = inter;
    *bytes = workspace_bytes_of(S, backward != 0);
    return MOE_SHUFFLE_OK;
}

int moe_experts_ffn_forward(moe_shuffle_plan_t plan, const void* xe, const void* w_gate_up, const void* w_down,
                            int32_t inter, int32_t act, void* ye, void* saved, void* saved_scale, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    ms::ExpertShape S;
    int rc = expert_shape(plan, inter, act, &S);
    if (rc) return rc;
    if (saved_scale && !saved) return MOE_SHUFFLE_E_INVALID_ARG;
    if (S.P == 0) return MOE_SHUFFLE_OK;
    if (!xe || !w_gate_up || !w_down || !ye) return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(xe, 16) || misaligned(w_gate_up, 16) || misaligned(w_down, 16) || misaligned(ye, 16) ||
        misaligned(saved, 16) || misaligned(saved_scale, 16))
        return MOE_SHUFFLE_E_ALIGN;
    rc = check_workspace(S, false, workspace, workspace_bytes);
    if (rc) return rc;
    const size_t rows = (size_t)S.P * S.H * 2, proj = (size_t)S.E * S.I * S.H * 2;
    if (overlaps({{ye, rows}, {saved, saved_bytes(S, saved_scale)}, {saved_scale, scale_bytes(S)},
                  {workspace, workspace_bytes_of(S, false)}},
                 {{xe, rows}, {w_gate_up, 2 * proj}, {w_down, proj}, plan_span(plan)}))
        return MOE_SHUFFLE_E_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    const bool few = ms::ffn_is_few(S);
    const ms::SavedActs held{saved, saved_scale};
    hipError_t e = few ? ms::launch_few_up(S, xe, w_gate_up, workspace, held, s)
                       : ms::launch_ffn_up(S, xe, w_gate_up, workspace, held, s);
    if (e == hipSuccess)
        e = few ? ms::launch_few_down(S, workspace, w_down, ye, s) : ms::launch_ffn_down(S, workspace, w_down, ye, s);
    return status_of(e);
}

int moe_experts_ffn_backward(moe_shuffle_plan_t plan, const void* grad_ye, const void* xe, const void* w_gate_up,
                             const void* w_down, int32_t inter, int32_t act, const void* saved,
                             const void* saved_scale, void* grad_xe, void* grad_w_gate_up, void* grad_w_down,
                             void* workspace, size_t workspace_bytes, void* stream)
{
    ms::ExpertShape S;
    int rc = expert_shape(plan, inter, act, &S);
    if (rc) return rc;
    // with no rows only the (zero) weight gradients are written, and nothing is read
    if (S.P > 0 && (!grad_ye || !w_down || !saved || (grad_xe && !w_gate_up) || (grad_w_gate_up && !xe)))
        return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(grad_ye, 16) || misaligned(xe, 16) || misaligned(w_gate_up, 16) || misaligned(w_down, 16) ||
        misaligned(saved, 16) || misaligned(saved_scale, 16) || misaligned(grad_xe, 16) ||
        misaligned(grad_w_gate_up, 16) || misaligned(grad_w_down, 16))
        return MOE_SHUFFLE_E_ALIGN;
    rc = check_workspace(S, true, workspace, workspace_bytes);
    if (rc) return rc;
    const size_t rows = (size_t)S.P * S.H * 2, proj = (size_t)S.E * S.I * S.H * 2;
    if (overlaps({{grad_xe, rows}, {grad_w_gate_up, 2 * proj}, {grad_w_down, proj},
                  {workspace, workspace_bytes_of(S, true)}},
                 {{grad_ye, rows}, {xe, rows}, {w_gate_up, 2 * proj}, {w_down, proj},
                  {saved, saved_bytes(S, saved_scale)}, {saved_scale, scale_bytes(S)}, plan_span(plan)}))
        return MOE_SHUFFLE_E_INVALID_ARG;
    if (!grad_xe && !grad_w_gate_up && !grad_w_down) return MOE_SHUFFLE_OK;
    hipStream_t s = (hipStream_t)stream;
    char* const h = (char*)workspace;
    char* const dgu = h + hidden_bytes(S);
    hipError_t e = hipSuccess;
    if (S.P > 0) {
        e = ms::launch_ffn_dh(S, grad_ye, w_down, ms::SavedActs{(void*)saved, (void*)saved_scale}, h, dgu, s);
        if (e == hipSuccess && grad_xe) e = ms::launch_ffn_dx(S, dgu, w_gate_up, grad_xe, s);
    }
    if (e == hipSuccess && grad_w_gate_up) e = ms::launch_ffn_wgrad(S, dgu, 2 * S.I, xe, S.H, grad_w_gate_up, s);
    if (e == hipSuccess && grad_w_down) e = ms::launch_ffn_wgrad(S, grad_ye, S.H, h, S.I, grad_w_down, s);
    return status_of(e);
}

int moe_experts_ffn_w4_forward(moe_shuffle_plan_t plan, const void* xe, const void* q_gate_up, const void* s_gate_up,
                               const void* q_down, const void* s_down, int32_t inter, int32_t group, int32_t act,
                               void* ye, void* workspace, size_t workspace_bytes, void* stream)
{
    ms::ExpertShape S;
    int rc = expert_shape(plan, inter, act, &S);
    if (rc) return rc;
    if (group != 32 && group != 64 && group != 128) return MOE_SHUFFLE_E_INVALID_ARG;
    if (S.H % group || S.I % group) return MOE_SHUFFLE_E_ALIGN;
    if (S.P == 0) return MOE_SHUFFLE_OK;
    if (!xe || !q_gate_up || !s_gate_up || !q_down || !s_down || !ye) return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(xe, 16) || misaligned(q_gate_up, 16) || misaligned(s_gate_up, 16) || misaligned(q_down, 16) ||
        misaligned(s_down, 16) || misaligned(ye, 16))
        return MOE_SHUFFLE_E_ALIGN;
    rc = check_workspace(S, false, workspace, workspace_bytes);
    if (rc) return rc;
    const size_t rows = (size_t)S.P * S.H * 2, proj = (size_t)S.E * S.I * S.H / 2;
    if (overlaps({{ye, rows}, {workspace, workspace_bytes_of(S, false)}},
                 {{xe, rows}, {q_gate_up, 2 * proj}, {q_down, proj}, {s_gate_up, 8 * proj / group},
                  {s_down, 4 * proj / group}, plan_span(plan)}))
        return MOE_SHUFFLE_E_INVALID_ARG;
    hipError_t e = ms::launch_w4_up(S, xe, q_gate_up, s_gate_up, group, workspace, (hipStream_t)stream);
    if (e == hipSuccess) e = ms::launch_w4_down(S, workspace, q_down, s_down, group, ye, (hipStream_t)stream);
    return status_of(e);
}

int moe_experts_w4_quantize(const void* w, int64_t rows, int32_t cols, int32_t group, void* q, void* scale,
                            void* stream)
{
    if (rows < 0 || cols <= 0 || (group != 32 && group != 64 && group != 128)) return MOE_SHUFFLE_E_INVALID_ARG;
    if (cols % group) return MOE_SHUFFLE_E_ALIGN;
    if (rows >= (int64_t)1 << 38 || rows * (cols / group) >= (int64_t)1 << 38) return MOE_SHUFFLE_E_OVERFLOW;
    if (rows == 0) return MOE_SHUFFLE_OK;
    if (!w || !q || !scale) return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(w, 16) || misaligned(q, 16) || misaligned(scale, 16)) return MOE_SHUFFLE_E_ALIGN;
    const size_t n = (size_t)rows * cols;
    if (overlaps({{q, n / 2}, {scale, 2 * (n / group)}}, {{w, 2 * n}})) return MOE_SHUFFLE_E_INVALID_ARG;
    return status_of(ms::launch_w4_quantize(w, rows, cols, group, q, scale, (hipStream_t)stream));
}

namespace {

int check_pack(const void* wide, const void* q, const void* scale, int64_t rows, int32_t cols)
{
    if (rows < 0 || cols <= 0) return MOE_SHUFFLE_E_INVALID_ARG;
    if (cols % 8) return MOE_SHUFFLE_E_ALIGN;
    const int64_t groups = ((int64_t)cols + ms::kGroup8 - 1) / ms::kGroup8;
    if (rows >= (int64_t)1 << 36 || rows * groups >= (int64_t)1 << 36) return MOE_SHUFFLE_E_OVERFLOW;
    if (rows == 0) return MOE_SHUFFLE_OK;
    if (!wide || !q || !scale) return MOE_SHUFFLE_E_INVALID_ARG;
    if (misaligned(wide, 16) || misaligned(q, 16) || misaligned(scale, 16)) return MOE_SHUFFLE_E_ALIGN;
    return MOE_SHUFFLE_OK;
}

}  // namespace

int moe_experts_pack8(const void* x, int64_t rows, int32_t cols, void* q, void* scale, void* stream)
{
    const int rc = check_pack(x, q, scale, rows, cols);
    if (rc || rows == 0) return rc;
    const size_t n = (size_t)rows * cols, groups = (size_t)rows * (((size_t)cols + ms::kGroup8 - 1) / ms::kGroup8);
    if (overlaps({{q, n}, {scale, 2 * groups}}, {{x, 2 * n}})) return MOE_SHUFFLE_E_INVALID_ARG;
    return status_of(ms::launch_pack8(x, rows, cols, q, scale, (hipStream_t)stream));
}

int moe_experts_unpack8(const void* q, const void* scale, int64_t rows, int32_t cols, void* x, void* stream)
{
    const int rc = check_pack(x, q, scale, rows, cols);
    if (rc || rows == 0) return rc;
    const size_t n = (size_t)rows * cols, groups = (size_t)rows * (((size_t)cols + ms::kGroup8 - 1) / ms::kGroup8);
    if (overlaps({{x, 2 * n}}, {{q, n}, {scale, 2 * groups}})) return MOE_SHUFFLE_E_INVALID_ARG;
    return status_of(ms::launch_unpack8(q, scale, rows, cols, x, (hipStream_t)stream));
}

}  // extern "C"
