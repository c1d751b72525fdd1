// optim.hip -- AdamW over many tensors at once, states in fp32 or in 8 bits (include/moe_optim.h has the formulas
// and the formats), and the way between 8-bit states and their values.
//
// Every element is read and written once, so the bytes are the bound: 28 an element with fp32 states, fp32
// parameters, their bf16 copy and bf16 gradients, 16.1 with 8-bit states.  What reaches the memory's rate is small
// blocks in the order of memory: with four neighbouring elements a lane (16 contiguous bytes of fp32) and 1024 a block,
// 197 M parameters with fp32 states take 910 us (6.1 TB/s, a large copy 6.5); 1028 with 8192 a block, 1128 with 8192 in
// lanes of eight.  8-bit states, 1.4 G parameters: 3.81 to 3.98 ms (6.0 to 5.8 TB/s) with 1024 a block of two waves, 4.07
// of four, 4.27 with 8192.  Unpacking moves fewer bytes an element and likes lanes of eight: 1.37 to 1.42 ms (6.2 to 6.0
// TB/s) against 1.57.  Packing 201 M fp32 values takes 354 us (5.7 TB/s).
//
// Rate and step that the device holds cost each thread two 64-bit powers, which the memory hides where states are fp32 (201 M
// parameters in a graph 898 us, 971 without) and not quite with 8 bits (620, 562).
//
// A group of 128 is 32 or 16 neighbouring lanes, which find its largest magnitudes by five or four exchanges.  The
// tensors' addresses come with the kernel's arguments, 40 a launch, so that nothing has to be copied to the device first.
#include <hip/hip_runtime.h>
#include <math.h>

#include <type_traits>

#include "checks.h"
#include "device_common.h"
#include "experts.h"
#include "moe_optim.h"

namespace ms {
namespace {

constexpr int kTensors = 40;  // of a launch
constexpr int kGroup = MOE_ADAMW_GROUP;
// Group steps are the largest magnitudes times these: the largest becomes 448 = 1.75 2^8 or 8064 = 63 2^7.
constexpr float kPerM = 1.0f / 448.0f, kPerS = 1.0f / 8064.0f;

// A kernel's blocks: Threads lanes of Each elements, Turns times.
template <int EACH, int THREADS, int TURNS>
struct Shape {
    static constexpr int kEach = EACH, kThreads = THREADS, kTurns = TURNS;
    static constexpr int kTurn = kEach * kThreads, kChunk = kTurn * kTurns;
    static constexpr int kLanes = kGroup / kEach;  // of a group
};
typedef Shape<4, 256, 1> StepWide;
typedef Shape<4, 128, 2> StepEight;
typedef Shape<8, 256, 1> Convert;

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

// ---- a lane's N elements (4 or 8) at i, of which `n` exist; the others read as zero ----

template <bool Half, int N>
__device__ __forceinline__ void read(const char* from, int64_t i, int n, float (&f)[N])
{
    if (n >= N) {
        if constexpr (Half) {
            typedef unsigned vec __attribute__((ext_vector_type(N / 2)));
            const vec d = __builtin_nontemporal_load((const vec*)(from + i * 2));
#pragma unroll
            for (int c = 0; c < N / 2; ++c) { f[2 * c] = bf16_lo(d[c]); f[2 * c + 1] = bf16_hi(d[c]); }
        } else {
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                const u32x4 a = __builtin_nontemporal_load((const u32x4*)(from + i * 4) + h);
#pragma unroll
                for (int c = 0; c < 4; ++c) f[4 * h + c] = __uint_as_float(a[c]);
            }
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < N; ++c)
        f[c] = c >= n ? 0.0f
               : Half ? __uint_as_float((unsigned)((const unsigned short*)from)[i + c] << 16)
                      : ((const float*)from)[i + c];
}

template <bool Half, int N>
__device__ __forceinline__ void write(char* to, int64_t i, int n, const float (&f)[N])
{
    if (n >= N) {
        if constexpr (Half) {
            typedef unsigned vec __attribute__((ext_vector_type(N / 2)));
            vec d;
#pragma unroll
            for (int c = 0; c < N / 2; ++c) d[c] = bf16_pack2(f[2 * c], f[2 * c + 1]);
            __builtin_nontemporal_store(d, (vec*)(to + i * 2));
        } else {
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                u32x4 a;
#pragma unroll
                for (int c = 0; c < 4; ++c) a[c] = __float_as_uint(f[4 * h + c]);
                __builtin_nontemporal_store(a, (u32x4*)(to + i * 4) + h);
            }
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < N; ++c)
        if (c < n) {
            if (Half) ((unsigned short*)to)[i + c] = (unsigned short)bf16_pack2(f[c], f[c]);
            else ((float*)to)[i + c] = f[c];
        }
}

// N codes, four a register.
template <int N>
struct Codes {
    typedef unsigned vec __attribute__((ext_vector_type(N / 4 == 1 ? 2 : N / 4)));
    unsigned d[N / 4];

    __device__ __forceinline__ void read(const char* from, int64_t i, int n)
    {
        if (n >= N) {
            if constexpr (N == 4) {
                d[0] = __builtin_nontemporal_load((const unsigned*)(from + i));
            } else {
                const vec v = __builtin_nontemporal_load((const vec*)(from + i));
                d[0] = v[0];
                d[1] = v[1];
            }
            return;
        }
#pragma unroll
        for (int h = 0; h < N / 4; ++h) d[h] = 0;
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (c < n) d[c >> 2] |= (unsigned)((const unsigned char*)from)[i + c] << (8 * (c & 3));
    }

    __device__ __forceinline__ void write(char* to, int64_t i, int n) const
    {
        if (n >= N) {
            if constexpr (N == 4) __builtin_nontemporal_store(d[0], (unsigned*)(to + i));
            else __builtin_nontemporal_store(vec{d[0], d[1]}, (vec*)(to + i));
            return;
        }
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (c < n) to[i + c] = (char)(d[c >> 2] >> (8 * (c & 3)));
    }
};

// ---- 8-bit states ----

template <int N>
__device__ __forceinline__ void values_m(const Codes<N>& q, float step, float (&f)[N])
{
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(q.d[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(q.d[h], true);
        f[4 * h] = a[0] * step;
        f[4 * h + 1] = a[1] * step;
        f[4 * h + 2] = b[0] * step;
        f[4 * h + 3] = b[1] * step;
    }
}

// Codes c > 0 of s: as the upper bits of a float, 32 2^(c / 32) has the exponent 5 + c / 32.
constexpr int kBaseS = 132 << 5;

template <int N>
__device__ __forceinline__ void values_s(const Codes<N>& q, float step, float (&f)[N])
{
#pragma unroll
    for (int c = 0; c < N; ++c) {
        const unsigned code = (q.d[c >> 2] >> (8 * (c & 3))) & 255u;
        f[c] = (code ? __uint_as_float((code + kBaseS) << 18) : 0.0f) * step;
    }
}

// The step of a group: its largest magnitude times `per`, at least 2^-126; NaN where one is not finite.
template <int N>
__device__ __forceinline__ float group_step(const float (&f)[N], float per)
{
    float most = 0;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        const float a = fabsf(f[c]);
        bad |= !(a <= 3.40282347e38f);
        most = fmaxf(most, a);
    }
    if (bad) most = __uint_as_float(0x7f800000u);
#pragma unroll
    for (int d = 1; d < kGroup / N; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, kWave));
    return most <= 3.40282347e38f ? fmaxf(most * per, 1.17549435e-38f) : __uint_as_float(0x7fc00000u);
}

// v_cvt_pk_fp8_f32: e4m3, to the nearest, the even one of two.  |f inv| is at most 448 (1 + 2^-23), which is 448.
template <int N>
__device__ __forceinline__ Codes<N> codes_m(const float (&f)[N], float step)
{
    Codes<N> q = {};
    if (step != step) return q;
    const float inv = 1.0f / step;
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * inv, f[4 * h + 1] * inv, 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * inv, f[4 * h + 3] * inv, v, true);
        q.d[h] = (unsigned)v;
    }
    return q;
}

template <int N>
__device__ __forceinline__ Codes<N> codes_s(const float (&f)[N], float step)
{
    Codes<N> q = {};
    if (step != step) return q;
    const float inv = 1.0f / step;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        const int u = __float_as_int(f[c] * inv);
        const int code = min(max(((u + 0x1ffff + ((u >> 18) & 1)) >> 18) - kBaseS, 1), 255);
        q.d[c >> 2] |= (f[c] > 0.0f ? (unsigned)code : 0u) << (8 * (c & 3));
    }
    return q;
}

// ---- the kernels ----

// The tensor of a chunk (its place in the launch; the same in every lane).
__device__ __forceinline__ int tensor_of(const Tensors& A, int chunk)
{
    const int lane = lane_id();
    return __builtin_ctzll(__ballot(lane < A.count && A.first[min(lane, kTensors - 1) + 1] > chunk));
}

// Calls f(i, n) for a block's turns: this lane's elements at i, n of them in the tensor (at least one in some lane of
// each wave that is called).
template <class B, class F>
__device__ __forceinline__ void turns(int64_t n, int chunk, F&& f)
{
    const int64_t at = (int64_t)chunk * B::kChunk + threadIdx.x * B::kEach;
#pragma unroll
    for (int turn = 0; turn < B::kTurns; ++turn) {
        const int64_t i = at + turn * B::kTurn, left = n - i;
        if (n - (i - lane_id() * B::kEach) <= 0) return;  // the same in every lane
        f(i, (int)(left < 0 ? 0 : left < B::kEach ? left : B::kEach));
    }
}

// The group of the lane's elements at i.
template <class B>
__device__ __forceinline__ int64_t group_of(int64_t i)
{
    return (i - (lane_id() & (B::kLanes - 1)) * B::kEach) / kGroup;
}

// Packs a lane's elements of states; every lane of a group calls it.
template <class B>
__device__ __forceinline__ void pack(const Tensor& t, int64_t i, int n, const float (&m)[B::kEach],
                                     const float (&s)[B::kEach])
{
    const float step_m = group_step(m, kPerM), step_s = group_step(s, kPerS);
    codes_m(m, step_m).write(t.m, i, n);
    codes_s(s, step_s).write(t.v, i, n);
    if ((lane_id() & (B::kLanes - 1)) == 0 && n > 0) {
        const int64_t group = group_of<B>(i);
        t.m_scale[group] = step_m;
        t.v_scale[group] = step_s;
    }
}

template <bool HalfP, bool HalfG, bool Eight, class B>
__global__ __launch_bounds__(B::kThreads) void adamw_kernel(Tensors A, Rates fixed, Hyper h)
{
    constexpr int N = B::kEach;
    const int which = tensor_of(A, blockIdx.x);
    const Tensor t = A.t[which];
    const int chunk = blockIdx.x - A.first[which];
    Rates r = fixed;
    if (h.lr_device || h.step_device) {
        const int64_t step = h.step_device ? *h.step_device : h.step;
        r = rates_of(h, h.lr_device ? (double)*h.lr_device : h.lr, step < 1 ? 1 : step);
    }
    const float scale = h.grad_scale ? *h.grad_scale : 1.0f;
    turns<B>(t.n, chunk, [&](int64_t i, int n) {
        float g[N], m[N], s[N], p[N];
        read<HalfG>(t.g, i, n, g);
        read<HalfP>(t.p, i, n, p);
        if constexpr (Eight) {
            const int64_t group = group_of<B>(i);
            const bool any = group * kGroup < t.n;
            Codes<N> qm, qs;
            qm.read(t.m, i, n);
            qs.read(t.v, i, n);
            values_m(qm, any ? t.m_scale[group] : 0.0f, m);
            values_s(qs, any ? t.v_scale[group] : 0.0f, s);
#pragma unroll
            for (int c = 0; c < N; ++c) s[c] *= s[c];
        } else {
            read<false>(t.m, i, n, m);
            read<false>(t.v, i, n, s);
        }
        float v[N];
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const float d = g[c] * scale;
            m[c] = m[c] * r.b1 + d * r.a1;
            v[c] = s[c] * r.b2 + d * d * r.a2;
            s[c] = sqrtf(v[c]);
            p[c] = p[c] * r.keep - r.gain * m[c] / (s[c] * r.root + r.eps);
        }
        write<HalfP>(t.p, i, n, p);
        if (!HalfP && t.copy) write<true>(t.copy, i, n, p);
        if constexpr (Eight) {
            if (n < N) {  // what is not there counts as zero
#pragma unroll
                for (int c = 0; c < N; ++c)
                    if (c >= n) m[c] = s[c] = 0.0f;
            }
            pack<B>(t, i, n, m, s);
        } else {
            write<false>(t.m, i, n, m);
            write<false>(t.v, i, n, v);
        }
    });
}

// p and copy hold m_out and v_out.
template <class B>
__global__ __launch_bounds__(B::kThreads) void adamw_pack_kernel(Tensors A)
{
    const int which = tensor_of(A, blockIdx.x);
    const Tensor t = A.t[which];
    turns<B>(t.n, blockIdx.x - A.first[which], [&](int64_t i, int n) {
        float m[B::kEach], s[B::kEach];
        read<false>(t.p, i, n, m);
        read<false>(t.copy, i, n, s);
#pragma unroll
        for (int c = 0; c < B::kEach; ++c) s[c] = s[c] < 0.0f ? 0.0f : sqrtf(s[c]);
        pack<B>(t, i, n, m, s);
    });
}

template <bool Half, class B>
__global__ __launch_bounds__(B::kThreads) void adamw_unpack_kernel(Tensors A)
{
    const int which = tensor_of(A, blockIdx.x);
    const Tensor t = A.t[which];
    turns<B>(t.n, blockIdx.x - A.first[which], [&](int64_t i, int n) {
        if (n <= 0) return;
        float m[B::kEach], s[B::kEach];
        const int64_t group = i / kGroup;
        Codes<B::kEach> qm, qs;
        qm.read(t.m, i, n);
        qs.read(t.v, i, n);
        values_m(qm, t.m_scale[group], m);
        values_s(qs, t.v_scale[group], s);
#pragma unroll
        for (int c = 0; c < B::kEach; ++c) s[c] *= s[c];
        write<Half>(t.p, i, n, m);
        write<Half>(t.copy, i, n, s);
    });
}

// ---- the boundary ----

size_t scale_bytes(int64_t n) { return (size_t)((n + kGroup - 1) / kGroup) * 4; }

enum class Call { Step, Pack, Unpack };

// Checks a call's tensors; p_size and the others are bytes an element.
int check_tensors(const moe_adamw_tensor* tensors, int32_t count, Call call, size_t p_size, size_t g_size, bool eight)
{
    if (count < 0 || (count > 0 && !tensors)) return MOE_SHUFFLE_E_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (t.n < 0) return MOE_SHUFFLE_E_INVALID_ARG;
        if (t.n >= (int64_t)1 << 40) return MOE_SHUFFLE_E_OVERFLOW;
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

// Bytes an element of what a call's kernel finds in a Tensor.
struct Sizes {
    int p, copy, g, state;
};

// launch(grid, tensors) for every 40 tensors that have an element; of one with very many, pieces of 2^32.
template <class B, class F>
hipError_t launch_tensors(const moe_adamw_tensor* tensors, int32_t count, bool step, const Sizes& size, F&& launch)
{
    constexpr int64_t kPiece = (int64_t)1 << 32;
    static_assert(kPiece % B::kChunk == 0 && kPiece % kGroup == 0, "pieces of whole chunks and groups");
    // one dispatch carries fewer than 2^32 work-items
    static_assert(kPiece / B::kChunk * B::kThreads < (int64_t)1 << 32, "a piece fits a dispatch");
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
        for (int64_t at = 0; at < t.n; at += kPiece) {
            const int64_t n = t.n - at < kPiece ? t.n - at : kPiece, more = (n + B::kChunk - 1) / B::kChunk;
            if (A.count == kTensors || (chunks + more) * B::kThreads >= (int64_t)1 << 32) {
                const hipError_t e = go();
                if (e != hipSuccess) return e;
            }
            const auto from = [&](const void* p, int bytes) { return p ? (char*)p + at * bytes : nullptr; };
            const auto scales = [&](float* p) { return p ? p + at / kGroup : nullptr; };
            A.t[A.count] = Tensor{from(step ? t.p : t.m_out, size.p),    from(step ? t.copy : t.v_out, size.copy),
                                  from(t.g, size.g),                     from(t.m, size.state),
                                  from(t.v, size.state),                 scales(t.m_scale),
                                  scales(t.v_scale),                     n};
            A.first[A.count++] = (int)chunks;
            chunks += more;
            A.first[A.count] = (int)chunks;
        }
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
    const Sizes size{half_p ? 2 : 4, 2, half_g ? 2 : 4, eight ? 1 : 4};
    const auto run = [&](auto p, auto g, auto e) {
        typedef std::conditional_t<decltype(e)::value, StepEight, StepWide> B;
        return status_of(launch_tensors<B>(tensors, count, true, size, [&](dim3 grid, const Tensors& A) {
            adamw_kernel<decltype(p)::value, decltype(g)::value, decltype(e)::value, B>
                <<<grid, B::kThreads, 0, s>>>(A, r, h);
        }));
    };
    const auto with_state = [&](auto p, auto g) {
        return eight ? run(p, g, std::true_type()) : run(p, g, std::false_type());
    };
    const auto with_grad = [&](auto p) {
        return half_g ? with_state(p, std::true_type()) : with_state(p, std::false_type());
    };
    return half_p ? with_grad(std::true_type()) : with_grad(std::false_type());
}

int moe_adamw_pack(const moe_adamw_tensor* tensors, int32_t count, void* stream)
{
    const int rc = check_tensors(tensors, count, Call::Pack, 4, 4, true);
    if (rc) return rc;
    return status_of(launch_tensors<Convert>(tensors, count, false, Sizes{4, 4, 0, 1}, [&](dim3 grid, const Tensors& A) {
        adamw_pack_kernel<Convert><<<grid, Convert::kThreads, 0, (hipStream_t)stream>>>(A);
    }));
}

int moe_adamw_unpack(const moe_adamw_tensor* tensors, int32_t count, int32_t values, void* stream)
{
    if (values != MOE_ADAMW_F32 && values != MOE_ADAMW_BF16) return MOE_SHUFFLE_E_INVALID_ARG;
    const bool half = values == MOE_ADAMW_BF16;
    const int rc = check_tensors(tensors, count, Call::Unpack, half ? 2 : 4, 4, true);
    if (rc) return rc;
    const Sizes size{half ? 2 : 4, half ? 2 : 4, 0, 1};
    return status_of(launch_tensors<Convert>(tensors, count, false, size, [&](dim3 grid, const Tensors& A) {
        if (half) adamw_unpack_kernel<true, Convert><<<grid, Convert::kThreads, 0, (hipStream_t)stream>>>(A);
        else adamw_unpack_kernel<false, Convert><<<grid, Convert::kThreads, 0, (hipStream_t)stream>>>(A);
    }));
}

}  // extern "C"
