// optim.hip -- AdamW over many tensors at once, states in fp32 or in 8 bits (include/moe_optim.h has the formulas
// and the formats), and the way between 8-bit states and their values.
//
// Every element is read and written once, so the bytes are the bound: 28 an element with fp32 states, fp32
// parameters, their bf16 copy and bf16 gradients, 16.1 with 8-bit states.  A lane has eight neighbouring elements
// (16 or 32 bytes of each kind), sixteen neighbouring lanes a group of 128, whose largest magnitudes four exchanges
// within the sixteen find.  A block takes 8192 elements of one tensor; the tensors' addresses come with the kernel's
// arguments, 40 a launch, so that nothing has to be copied to the device first.
#include <hip/hip_runtime.h>
#include <math.h>

#include "checks.h"
#include "device_common.h"
#include "experts.h"
#include "moe_optim.h"

namespace ms {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 8;                    // elements of a lane
constexpr int kTurn = kThreads * kEach;     // elements a block has at once
constexpr int kChunk = 4 * kTurn;           // of a block
constexpr int kTensors = 40;                // of a launch
constexpr int kGroup = MOE_ADAMW_GROUP;
// Group steps are the largest magnitudes times these: the largest becomes 448 = 1.75 2^8 or 8064 = 63 2^7.
constexpr float kPerM = 1.0f / 448.0f, kPerS = 1.0f / 8064.0f;
static_assert(kGroup == 16 * kEach, "sixteen lanes a group");

struct Tensor {
    char *p, *copy;
    const char* g;
    char *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
};

struct Tensors {
    Tensor t[kTensors];
    int first[kTensors + 1];  // chunk of each tensor
    int count;
};

// The constants of a step.
struct Rates {
    float b1, a1, b2, a2, eps;  // a = 1 - b
    float keep, gain, root;     // 1 - lr weight_decay, lr / (1 - b1^step), 1 / sqrt(1 - b2^step)
};

struct Hyper {
    double lr, b1, b2, eps, decay;
    int64_t step;
    const float* lr_device;
    const int64_t* step_device;
    const float* grad_scale;
};

__host__ __device__ inline double power(double b, int64_t n)
{
    double r = 1;
    for (; n > 0; n >>= 1) {
        if (n & 1) r *= b;
        b *= b;
    }
    return r;
}

__host__ __device__ inline Rates rates_of(const Hyper& h, double lr, int64_t step)
{
    Rates r;
    r.b1 = (float)h.b1;
    r.a1 = (float)(1 - h.b1);
    r.b2 = (float)h.b2;
    r.a2 = (float)(1 - h.b2);
    r.eps = (float)h.eps;
    r.keep = (float)(1 - lr * h.decay);
    r.gain = (float)(lr / (1 - power(h.b1, step)));
    r.root = (float)(1 / sqrt(1 - power(h.b2, step)));
    return r;
}

// ---- a lane's eight elements at i, of which `n` exist; the others read as zero ----

template <bool Half>
__device__ __forceinline__ void read8(const char* from, int64_t i, int n, float (&f)[kEach])
{
    if (n >= kEach) {
        if constexpr (Half) {
            const u32x4 d = __builtin_nontemporal_load((const u32x4*)(from + i * 2));
#pragma unroll
            for (int c = 0; c < 4; ++c) { f[2 * c] = bf16_lo(d[c]); f[2 * c + 1] = bf16_hi(d[c]); }
        } else {
            const u32x4 a = __builtin_nontemporal_load((const u32x4*)(from + i * 4));
            const u32x4 b = __builtin_nontemporal_load((const u32x4*)(from + i * 4) + 1);
#pragma unroll
            for (int c = 0; c < 4; ++c) { f[c] = __uint_as_float(a[c]); f[4 + c] = __uint_as_float(b[c]); }
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < kEach; ++c)
        f[c] = c >= n ? 0.0f
               : Half ? __uint_as_float((unsigned)((const unsigned short*)from)[i + c] << 16)
                      : ((const float*)from)[i + c];
}

template <bool Half>
__device__ __forceinline__ void write8(char* to, int64_t i, int n, const float (&f)[kEach])
{
    if (n >= kEach) {
        if constexpr (Half) {
            const u32x4 d = {bf16_pack2(f[0], f[1]), bf16_pack2(f[2], f[3]), bf16_pack2(f[4], f[5]),
                             bf16_pack2(f[6], f[7])};
            __builtin_nontemporal_store(d, (u32x4*)(to + i * 2));
        } else {
            u32x4 a, b;
#pragma unroll
            for (int c = 0; c < 4; ++c) { a[c] = __float_as_uint(f[c]); b[c] = __float_as_uint(f[4 + c]); }
            __builtin_nontemporal_store(a, (u32x4*)(to + i * 4));
            __builtin_nontemporal_store(b, (u32x4*)(to + i * 4) + 1);
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < kEach; ++c)
        if (c < n) {
            if (Half) ((unsigned short*)to)[i + c] = (unsigned short)bf16_pack2(f[c], f[c]);
            else ((float*)to)[i + c] = f[c];
        }
}

__device__ __forceinline__ u32x2 read_codes(const char* from, int64_t i, int n)
{
    if (n >= kEach) return __builtin_nontemporal_load((const u32x2*)(from + i));
    u32x2 d = {0, 0};
#pragma unroll
    for (int c = 0; c < kEach; ++c)
        if (c < n) d[c >> 2] |= (unsigned)((const unsigned char*)from)[i + c] << (8 * (c & 3));
    return d;
}

__device__ __forceinline__ void write_codes(char* to, int64_t i, int n, u32x2 d)
{
    if (n >= kEach) {
        __builtin_nontemporal_store(d, (u32x2*)(to + i));
        return;
    }
#pragma unroll
    for (int c = 0; c < kEach; ++c)
        if (c < n) to[i + c] = (char)(d[c >> 2] >> (8 * (c & 3)));
}

// ---- 8-bit states ----

__device__ __forceinline__ void values_m(u32x2 d, float step, float (&f)[kEach])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(d[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(d[h], true);
        f[4 * h] = a[0] * step;
        f[4 * h + 1] = a[1] * step;
        f[4 * h + 2] = b[0] * step;
        f[4 * h + 3] = b[1] * step;
    }
}

// Codes c > 0 of s: as the upper bits of a float, 32 2^(c / 32) has the exponent 5 + c / 32.
constexpr int kBaseS = 132 << 5;

__device__ __forceinline__ void values_s(u32x2 d, float step, float (&f)[kEach])
{
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
        const unsigned code = (d[c >> 2] >> (8 * (c & 3))) & 255u;
        f[c] = (code ? __uint_as_float((code + kBaseS) << 18) : 0.0f) * step;
    }
}

// The step of a group: its largest magnitude times `per`, at least 2^-126; NaN where one is not finite.
__device__ __forceinline__ float group_step(const float (&f)[kEach], float per)
{
    float most = 0;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
        const float a = fabsf(f[c]);
        bad |= !(a <= 3.40282347e38f);
        most = fmaxf(most, a);
    }
    if (bad) most = __uint_as_float(0x7f800000u);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, kWave));
    return most <= 3.40282347e38f ? fmaxf(most * per, 1.17549435e-38f) : __uint_as_float(0x7fc00000u);
}

// v_cvt_pk_fp8_f32: e4m3, to the nearest, the even one of two.  |f inv| is at most 448 (1 + 2^-23), which is 448.
__device__ __forceinline__ u32x2 codes_m(const float (&f)[kEach], float step)
{
    if (step != step) return u32x2{0, 0};
    const float inv = 1.0f / step;
    u32x2 d;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * inv, f[4 * h + 1] * inv, 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * inv, f[4 * h + 3] * inv, v, true);
        d[h] = (unsigned)v;
    }
    return d;
}

__device__ __forceinline__ u32x2 codes_s(const float (&f)[kEach], float step)
{
    if (step != step) return u32x2{0, 0};
    const float inv = 1.0f / step;
    u32x2 d = {0, 0};
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
        const int u = __float_as_int(f[c] * inv);
        const int code = min(max(((u + 0x1ffff + ((u >> 18) & 1)) >> 18) - kBaseS, 1), 255);
        d[c >> 2] |= (f[c] > 0.0f ? (unsigned)code : 0u) << (8 * (c & 3));
    }
    return d;
}

// ---- the kernels ----

// The tensor of a chunk (its place in the launch; the same in every lane).
__device__ __forceinline__ int tensor_of(const Tensors& A, int chunk)
{
    const int lane = lane_id();
    return __builtin_ctzll(__ballot(lane < A.count && A.first[min(lane, kTensors - 1) + 1] > chunk));
}

// Calls f(i, n) for a block's turns: this lane's eight elements at i, n of them in the tensor (at least one in some
// lane of each wave that is called).
template <class F>
__device__ __forceinline__ void turns(int64_t n, int chunk, F&& f)
{
    const int64_t at = (int64_t)chunk * kChunk + threadIdx.x * kEach;
#pragma unroll 1
    for (int turn = 0; turn < kChunk / kTurn; ++turn) {
        const int64_t i = at + turn * kTurn, left = n - i;
        if (n - (i - lane_id() * kEach) <= 0) return;  // the same in every lane
        f(i, (int)(left < 0 ? 0 : left < kEach ? left : kEach));
    }
}

template <bool HalfP, bool HalfG, bool Eight>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Tensors A, Rates fixed, Hyper h)
{
    const int which = tensor_of(A, blockIdx.x);
    const Tensor t = A.t[which];
    const int chunk = blockIdx.x - A.first[which];
    Rates r = fixed;
    if (h.lr_device || h.step_device) {
        const int64_t step = h.step_device ? *h.step_device : h.step;
        r = rates_of(h, h.lr_device ? (double)*h.lr_device : h.lr, step < 1 ? 1 : step);
    }
    const float scale = h.grad_scale ? *h.grad_scale : 1.0f;
    turns(t.n, chunk, [&](int64_t i, int n) {
        float g[kEach], m[kEach], s[kEach], p[kEach];
        read8<HalfG>(t.g, i, n, g);
        read8<HalfP>(t.p, i, n, p);
        if constexpr (Eight) {
            const int64_t group = (i - (lane_id() & 15) * kEach) / kGroup;
            const bool any = group * kGroup < t.n;
            values_m(read_codes(t.m, i, n), any ? t.m_scale[group] : 0.0f, m);
            values_s(read_codes(t.v, i, n), any ? t.v_scale[group] : 0.0f, s);
#pragma unroll
            for (int c = 0; c < kEach; ++c) s[c] *= s[c];
        } else {
            read8<false>(t.m, i, n, m);
            read8<false>(t.v, i, n, s);
        }
        float v[kEach];
#pragma unroll
        for (int c = 0; c < kEach; ++c) {
            const float d = g[c] * scale;
            m[c] = m[c] * r.b1 + d * r.a1;
            v[c] = s[c] * r.b2 + d * d * r.a2;
            s[c] = sqrtf(v[c]);
            p[c] = p[c] * r.keep - r.gain * m[c] / (s[c] * r.root + r.eps);
        }
        write8<HalfP>(t.p, i, n, p);
        if (!HalfP && t.copy) write8<true>(t.copy, i, n, p);
        if constexpr (Eight) {
            const int64_t group = (i - (lane_id() & 15) * kEach) / kGroup;
            if (n < kEach) {  // what is not there counts as zero (a gradient of zero leaves 0 unless eps is 0)
#pragma unroll
                for (int c = 0; c < kEach; ++c)
                    if (c >= n) m[c] = s[c] = 0.0f;
            }
            const float step_m = group_step(m, kPerM), step_s = group_step(s, kPerS);
            write_codes(t.m, i, n, codes_m(m, step_m));
            write_codes(t.v, i, n, codes_s(s, step_s));
            if ((lane_id() & 15) == 0 && n > 0) {
                t.m_scale[group] = step_m;
                t.v_scale[group] = step_s;
            }
        } else {
            write8<false>(t.m, i, n, m);
            write8<false>(t.v, i, n, v);
        }
    });
}

// p and copy hold m_out and v_out.
__global__ __launch_bounds__(kThreads) void adamw_pack_kernel(Tensors A)
{
    const int which = tensor_of(A, blockIdx.x);
    const Tensor t = A.t[which];
    turns(t.n, blockIdx.x - A.first[which], [&](int64_t i, int n) {
        float m[kEach], s[kEach];
        read8<false>(t.p, i, n, m);
        read8<false>(t.copy, i, n, s);
#pragma unroll
        for (int c = 0; c < kEach; ++c) s[c] = s[c] < 0.0f ? 0.0f : sqrtf(s[c]);
        const int64_t group = (i - (lane_id() & 15) * kEach) / kGroup;
        const float step_m = group_step(m, kPerM), step_s = group_step(s, kPerS);
        write_codes(t.m, i, n, codes_m(m, step_m));
        write_codes(t.v, i, n, codes_s(s, step_s));
        if ((lane_id() & 15) == 0 && n > 0) {
            t.m_scale[group] = step_m;
            t.v_scale[group] = step_s;
        }
    });
}

template <bool Half>
__global__ __launch_bounds__(kThreads) void adamw_unpack_kernel(Tensors A)
{
    const int which = tensor_of(A, blockIdx.x);
    const Tensor t = A.t[which];
    turns(t.n, blockIdx.x - A.first[which], [&](int64_t i, int n) {
        if (n <= 0) return;
        float m[kEach], s[kEach];
        const int64_t group = i / kGroup;
        values_m(read_codes(t.m, i, n), t.m_scale[group], m);
        values_s(read_codes(t.v, i, n), t.v_scale[group], s);
#pragma unroll
        for (int c = 0; c < kEach; ++c) s[c] *= s[c];
        write8<Half>(t.p, i, n, m);
        write8<Half>(t.copy, i, n, s);
    });
}

// ---- the boundary ----

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }

size_t scale_bytes(int64_t n) { return (size_t)((n + kGroup - 1) / kGroup) * 4; }

enum class Call { Step, Pack, Unpack };

// Checks a call's tensors; p_size and the others are bytes an element.
int check_tensors(const moe_adamw_tensor* tensors, int32_t count, Call call, size_t p_size, size_t g_size, bool eight)
{
    if (count < 0 || (count > 0 && !tensors)) return MOE_SHUFFLE_E_INVALID_ARG;
    int64_t chunks = 0;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (t.n < 0) return MOE_SHUFFLE_E_INVALID_ARG;
        if (t.n >= (int64_t)1 << 40 || (chunks += chunks_of(t.n)) >= (int64_t)1 << 31) return MOE_SHUFFLE_E_OVERFLOW;
        if (t.n == 0) continue;
        const bool step = call == Call::Step;
        const void* const a = step ? t.p : t.m_out;
        const void* const b = step ? t.g : t.v_out;
        if (!a || !b || !t.m || !t.v || (eight && (!t.m_scale || !t.v_scale))) return MOE_SHUFFLE_E_INVALID_ARG;
        if (step && t.copy && p_size != 4) return MOE_SHUFFLE_E_INVALID_ARG;
        const void* const copy = step ? t.copy : nullptr;
        if (misaligned(a, 16) || misaligned(b, 16) || misaligned(copy, 16) || misaligned(t.m, 16) ||
            misaligned(t.v, 16) || (eight && (misaligned(t.m_scale, 4) || misaligned(t.v_scale, 4))))
            return MOE_SHUFFLE_E_ALIGN;
        const size_t n = (size_t)t.n, state = eight ? n : 4 * n, sc = eight ? scale_bytes(t.n) : 0;
        const Span m{t.m, state}, v{t.v, state}, ms{t.m_scale, sc}, vs{t.v_scale, sc};
        const bool hit = step ? overlaps({{t.p, p_size * n}, {copy, 2 * n}, m, v, ms, vs}, {{t.g, g_size * n}})
                         : call == Call::Pack
                             ? overlaps({m, v, ms, vs}, {{t.m_out, p_size * n}, {t.v_out, p_size * n}})
                             : overlaps({{t.m_out, p_size * n}, {t.v_out, p_size * n}}, {m, v, ms, vs});
        if (hit) return MOE_SHUFFLE_E_INVALID_ARG;
    }
    return MOE_SHUFFLE_OK;
}

// launch(grid, tensors) for every 40 tensors that have an element.
template <class F>
hipError_t launch_tensors(const moe_adamw_tensor* tensors, int32_t count, bool step, F&& launch)
{
    Tensors A;
    A.count = 0;
    int64_t chunks = 0;
    const auto go = [&]() {
        if (!A.count) return hipSuccess;
        launch(dim3((unsigned)chunks), A);
        A.count = 0;
        chunks = 0;
        return hipGetLastError();
    };
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        // one dispatch carries fewer than 2^32 work-items
        if (A.count == kTensors || (chunks + chunks_of(t.n)) * kThreads >= (int64_t)1 << 32) {
            const hipError_t e = go();
            if (e != hipSuccess) return e;
        }
        A.t[A.count] = Tensor{(char*)(step ? t.p : t.m_out), (char*)(step ? t.copy : t.v_out), (const char*)t.g,
                              (char*)t.m, (char*)t.v, t.m_scale, t.v_scale, t.n};
        A.first[A.count++] = (int)chunks;
        chunks += chunks_of(t.n);
        A.first[A.count] = (int)chunks;
    }
    return go();
}

bool in_range(double v, double lo) { return v >= lo && v <= 1.7976931348623157e308; }

}  // namespace
}  // namespace ms

using namespace ms;

extern "C" {

int moe_adamw_step(const moe_adamw_tensor* tensors, int32_t count, const moe_adamw_params* q, void* stream)
{
    if (!q || q->reserved != 0) return MOE_SHUFFLE_E_INVALID_ARG;
    if ((q->param != MOE_ADAMW_F32 && q->param != MOE_ADAMW_BF16) ||
        (q->grad != MOE_ADAMW_F32 && q->grad != MOE_ADAMW_BF16) ||
        (q->state != MOE_ADAMW_F32 && q->state != MOE_ADAMW_8BIT))
        return MOE_SHUFFLE_E_INVALID_ARG;
    if (!in_range(q->lr, 0) || !in_range(q->eps, 0) || !in_range(q->weight_decay, 0) || !in_range(q->beta1, 0) ||
        !in_range(q->beta2, 0) || q->beta1 >= 1 || q->beta2 >= 1 || (q->step < 1 && !q->step_device))
        return MOE_SHUFFLE_E_INVALID_ARG;
    const bool half_p = q->param == MOE_ADAMW_BF16, half_g = q->grad == MOE_ADAMW_BF16;
    const bool eight = q->state == MOE_ADAMW_8BIT;
    if (misaligned(q->lr_device, 4) || misaligned(q->step_device, 8) || misaligned(q->grad_scale, 4))
        return MOE_SHUFFLE_E_ALIGN;
    const int rc = check_tensors(tensors, count, Call::Step, half_p ? 2 : 4, half_g ? 2 : 4, eight);
    if (rc) return rc;
    const Hyper h{q->lr, q->beta1, q->beta2, q->eps, q->weight_decay, q->step, q->lr_device, q->step_device,
                  q->grad_scale};
    const Rates r = rates_of(h, h.lr, h.step < 1 ? 1 : h.step);
    hipStream_t s = (hipStream_t)stream;
    return status_of(launch_tensors(tensors, count, true, [&](dim3 grid, const Tensors& A) {
        const auto go = [&](auto p, auto g, auto e) {
            adamw_kernel<decltype(p)::value, decltype(g)::value, decltype(e)::value><<<grid, kThreads, 0, s>>>(A, r, h);
        };
        const auto with_state = [&](auto p, auto g) {
            if (eight) go(p, g, std::true_type());
            else go(p, g, std::false_type());
        };
        const auto with_grad = [&](auto p) {
            if (half_g) with_state(p, std::true_type());
            else with_state(p, std::false_type());
        };
        if (half_p) with_grad(std::true_type());
        else with_grad(std::false_type());
    }));
}

int moe_adamw_pack(const moe_adamw_tensor* tensors, int32_t count, void* stream)
{
    const int rc = check_tensors(tensors, count, Call::Pack, 4, 4, true);
    if (rc) return rc;
    return status_of(launch_tensors(tensors, count, false, [&](dim3 grid, const Tensors& A) {
        adamw_pack_kernel<<<grid, kThreads, 0, (hipStream_t)stream>>>(A);
    }));
}

int moe_adamw_unpack(const moe_adamw_tensor* tensors, int32_t count, int32_t values, void* stream)
{
    if (values != MOE_ADAMW_F32 && values != MOE_ADAMW_BF16) return MOE_SHUFFLE_E_INVALID_ARG;
    const bool half = values == MOE_ADAMW_BF16;
    const int rc = check_tensors(tensors, count, Call::Unpack, half ? 2 : 4, 4, true);
    if (rc) return rc;
    return status_of(launch_tensors(tensors, count, false, [&](dim3 grid, const Tensors& A) {
        if (half) adamw_unpack_kernel<true><<<grid, kThreads, 0, (hipStream_t)stream>>>(A);
        else adamw_unpack_kernel<false><<<grid, kThreads, 0, (hipStream_t)stream>>>(A);
    }));
}

}  // extern "C"
