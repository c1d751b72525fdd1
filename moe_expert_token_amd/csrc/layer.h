// layer.h -- what the router's and the layer's files share (library-internal;
// the ABI is include/moe_layer.h): the routing rule, keys in 64 bits, and the
// choice of the largest by one wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "experts.h"
#include "moe_layer.h"

namespace ms {

constexpr int kLayerTokens = MOE_LAYER_MAX_TOKENS, kLayerPairs = MOE_LAYER_MAX_PAIRS;

struct Rule {
    int sigmoid, normalize;
    float scale;
    const float* bias;  // [E], sigmoid only
};

struct RouterShape {
    int T, H, E, k;
};

// A layer's call, and where its workspace keeps what.
struct LayerShape {
    int T, H, E, k, I, P;    // P = T k
    float c0, c1;            // the gate's sigmoid argument: c0 g + c1 g^3
    unsigned long long* key;  // [T][E], ordered_key of each expert's key
    float* logit;             // [T][E]
    int4* tile;               // [<= P] expert, first row, rows; rows are in the order of experts, then tokens
    int* tiles;               // [1] how many
    int* row_of;              // [P] the row of (token, slot)
    float* gate;              // [P]
    int* arrived;             // [ceil(H / 64)]
    char* h;                  // [P][I] bf16
    float* y;                 // [P][H]
};

size_t layer_workspace(LayerShape* S, char* base);

struct LayerCall {
    const void *x, *w_router, *up, *up_scale, *down, *down_scale, *residual;
    void* out;
    int32_t* topk_idx;
    float* topk_w;
    int group;  // 0: bf16 weights
};

hipError_t launch_layer(const LayerShape& S, const Rule& rule, const LayerCall& C, hipStream_t s);

size_t router_workspace(const RouterShape& S, bool backward);
hipError_t launch_router_forward(const RouterShape& S, const Rule& rule, const void* x, const void* w, int32_t* idx,
                                 float* gate, float* logits, char* ws, hipStream_t s);
hipError_t launch_router_backward(const RouterShape& S, const Rule& rule, const float* grad_gate, const float* logits,
                                  const int32_t* idx, const void* x, const void* w, const float* grad_logits,
                                  const void* grad_x_in, void* grad_x, void* grad_w, char* ws, hipStream_t s);

// ---- device helpers ----

// Keys as unsigned numbers of the same order; NaN as minus infinity, -0 as 0.  All are above 0, which stands for none.
__device__ __forceinline__ unsigned long long ordered_key(double v)
{
    if (v != v) v = -__builtin_inf();
    v += 0.0;
    const unsigned long long u = (unsigned long long)__double_as_longlong(v);
    return u >> 63 ? ~u : u | 1ull << 63;
}

__device__ __forceinline__ double score64(double l) { return 1.0 / (1.0 + exp(-l)); }

// The sums in 64 bits that the choice of experts goes by have one order, whichever kernel makes them, so that a token is
// routed alike by all calls also where products span more than 53 bits and the sum depends on their order: vectors of
// eight k are dealt to kSumParts parts of a wave each (vector v: lane v % 64 of part v / 64 % 8), a lane adds its products
// in the order of k, the lanes of a part are added those 32 apart first, then 16, 8, 4, 2, 1, and the parts in turn.
constexpr int kSumParts = 8;

// A double by its two registers.
union Halves {
    double d;
    unsigned u[2];
};

// a and b so that their sum is, in the lower of each two groups of D lanes, a's of both groups, in the upper b's.
template <int D>
__device__ __forceinline__ void exchange(double& a, double& b)
{
    Halves x, y;
    x.d = a;
    y.d = b;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (D == 32) {
            const auto r = __builtin_amdgcn_permlane32_swap(x.u[i], y.u[i], false, false);
            x.u[i] = r[0];
            y.u[i] = r[1];
        } else if constexpr (D == 16) {
            const auto r = __builtin_amdgcn_permlane16_swap(x.u[i], y.u[i], false, false);
            x.u[i] = r[0];
            y.u[i] = r[1];
        } else {
            const bool upper = lane_id() & D;
            const unsigned keep = upper ? y.u[i] : x.u[i], give = upper ? x.u[i] : y.u[i];
            x.u[i] = keep;
            y.u[i] = __shfl_xor(give, D, kWave);
        }
    }
    a = x.d;
    b = y.d;
}

// The value of the lane D further on in a row of sixteen, around its end.
template <int D>
__device__ __forceinline__ double turned(double v)
{
    Halves x;
    x.d = v;
#pragma unroll
    for (int i = 0; i < 2; ++i) x.u[i] = (unsigned)__builtin_amdgcn_update_dpp(0, (int)x.u[i], 0x120 + D, 0xf, 0xf, false);
    return x.d;
}

// The wave's sums of N values a lane (a power of two, up to 32): each exchange halves the values that a lane is left
// with, so that N + 5 or so of them do it and not 6 N.  Leaves one sum; returns which: the upper bits of the lane, so
// the first of 64 / N lanes each.
template <int N, int D = kWave / 2>
__device__ __forceinline__ int wave_sums(double (&v)[N], double* sum)
{
    if constexpr (N == 1) {
        double a = v[0];
        if constexpr (D >= 16) {  // both are `a`: the sum is the same in both groups
            double b = a;
            exchange<D>(a, b);
            double more[1] = {a + b};
            return wave_sums<1, D / 2>(more, sum);
        } else if constexpr (D == 8) {
            // the partner is that many lanes on: what comes out repeats itself as often in the row
            a += turned<8>(a);
            a += turned<4>(a);
            a += turned<2>(a);
            a += turned<1>(a);
        } else {
#pragma unroll
            for (int d = D; d > 0; d >>= 1) a += __shfl_xor(a, d, kWave);
        }
        *sum = a;
        return 0;
    } else {
        double half[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            double a = v[i], b = v[i + N / 2];
            exchange<D>(a, b);
            half[i] = a + b;
        }
        return (lane_id() & D ? N / 2 : 0) + wave_sums<N / 2, D / 2>(half, sum);
    }
}

__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

__device__ __forceinline__ double lane_value(double v, int lane)
{
    Halves x;
    x.d = v;
#pragma unroll
    for (int i = 0; i < 2; ++i) x.u[i] = (unsigned)__builtin_amdgcn_readlane((int)x.u[i], lane);
    return x.d;
}

template <class Part>
__device__ __forceinline__ double parts_total(Part&& part)
{
    double l = 0;
#pragma unroll
    for (int i = 0; i < kSumParts; ++i) l += part(i);
    return l;
}

template <int Ctrl, int Rows>
__device__ __forceinline__ unsigned dpp_max(unsigned v)
{
    return max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, Ctrl, Rows, 0xf, false));
}

// The largest of the wave's values (the same in every lane): within sixteens, then across them, without LDS.
__device__ __forceinline__ unsigned wave_max(unsigned v)
{
    v = dpp_max<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8: lane 15 of each row has the row's
    v = dpp_max<0x112, 0xf>(v);
    v = dpp_max<0x114, 0xf>(v);
    v = dpp_max<0x118, 0xf>(v);
    v = dpp_max<0x142, 0xa>(v);  // row_bcast 15 and 31
    v = dpp_max<0x143, 0xc>(v);
    return (unsigned)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
    return v;
}

__device__ __forceinline__ float wave_total(float v)
{
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
    return v;
}

// Inclusive scan over the wave, likewise.
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
    return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
}

// The place of the wave's largest of `key` (one a lane, with its index `at`); of equal ones the lowest index.
__device__ __forceinline__ int wave_argmax(unsigned long long key, int at)
{
    const unsigned hi = (unsigned)(key >> 32), lo = (unsigned)key;
    const unsigned top = wave_max(hi);
    unsigned long long m = __ballot(hi == top);
    if ((m & (m - 1)) == 0) return __builtin_amdgcn_readlane(at, __builtin_ctzll(m));
    const unsigned low = wave_max(hi == top ? lo : 0u);
    const bool one = hi == top && lo == low;
    m = __ballot(one);
    if ((m & (m - 1)) == 0) return __builtin_amdgcn_readlane(at, __builtin_ctzll(m));
    return (int)~wave_max(one ? ~(unsigned)at : 0u);
}

// The gates of a token: lane j < k has the logit l of slot j; `most` is the row's largest logit and `all` the sum of
// exp(logit - most) over the row, which softmax without normalization needs.
__device__ __forceinline__ float gate_of(const Rule& rule, int k, float l, float most, float all)
{
    const bool in = lane_id() < k;
    float s;
    if (rule.sigmoid) s = 1.0f / (1.0f + expf(-l));
    else s = expf(l - most) / (rule.normalize ? 1.0f : all);
    if (!in) s = 0.0f;
    if (rule.normalize) s = s / (wave_total(s) + 1e-20f);
    return rule.scale * s;
}

}  // namespace ms
