// experts.h -- launchers and device helpers shared by the files of the
// experts' block (library-internal; the ABI is include/moe_experts.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "device_common.h"
#include "moe_experts.h"

namespace ms {

constexpr int kGroup8 = MOE_EXPERTS_GROUP8;

// One block's shape and where the plan keeps its segments.
struct ExpertShape {
    int P, H, I, E;           // expert rows, widths, experts
    float c0, c1;             // the gate's sigmoid argument: c0 g + c1 g^3
    const int32_t* offset;    // [E + 1], device
    const int32_t* status;    // device; nonzero: write nothing
};

// The pre-activations held for the backward pass: bf16 (scale null) or int8.
struct SavedActs {
    void* data;
    void* scale;
};

// Each launcher returns the hipError_t of its launches.
hipError_t launch_ffn_up(const ExpertShape& S, const void* xe, const void* w_gate_up, void* h, SavedActs saved,
                         hipStream_t s);
hipError_t launch_ffn_down(const ExpertShape& S, const void* h, const void* w_down, void* ye, hipStream_t s);
hipError_t launch_ffn_dh(const ExpertShape& S, const void* grad_ye, const void* w_down, SavedActs saved, void* h,
                         void* dgu, hipStream_t s);
hipError_t launch_ffn_dx(const ExpertShape& S, const void* dgu, const void* w_gate_up, void* grad_xe, hipStream_t s);
// out[e] = a_e^T b_e over the rows of expert e: a [P, na], b [P, nb], out [E, na, nb].
hipError_t launch_ffn_wgrad(const ExpertShape& S, const void* a, int na, const void* b, int nb, void* out,
                            hipStream_t s);

// The forward pass where the experts have few rows each (ffn_is_few says when it is the faster one).
bool ffn_is_few(const ExpertShape& S);
hipError_t launch_few_up(const ExpertShape& S, const void* xe, const void* w_gate_up, void* h, SavedActs saved,
                         hipStream_t s);
hipError_t launch_few_down(const ExpertShape& S, const void* h, const void* w_down, void* ye, hipStream_t s);

hipError_t launch_w4_up(const ExpertShape& S, const void* xe, const void* q, const void* scale, int group, void* h,
                        hipStream_t s);
hipError_t launch_w4_down(const ExpertShape& S, const void* h, const void* q, const void* scale, int group, void* ye,
                          hipStream_t s);
hipError_t launch_w4_quantize(const void* w, int64_t rows, int cols, int group, void* q, void* scale, hipStream_t s);

hipError_t launch_pack8(const void* x, int64_t rows, int cols, void* q, void* scale, hipStream_t s);
hipError_t launch_unpack8(const void* q, const void* scale, int64_t rows, int cols, void* x, hipStream_t s);

// ---- device helpers ----

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_lo(unsigned u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) { return __uint_as_float(u & 0xffff0000u); }

// Two fp32 values rounded to nearest even bf16 ones (v_cvt_pk_bf16_f32; NaN stays NaN).
__device__ __forceinline__ unsigned bf16_pack2(float a, float b)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ f32x4 mfma_16x16x32(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// sigmoid(a(g)) and a'(g) of the gate.  The cubic is taken at g clamped to
// +-64, where the sigmoid has long reached 0 or 1, so that neither its square
// nor 0 * infinity (c1 = 0) can make a NaN of a finite g.
__device__ __forceinline__ float gate_sigmoid(float g, float c0, float c1, float* slope)
{
    const float t = fminf(fmaxf(g, -64.0f), 64.0f), t2 = t * t;
    *slope = fmaf(3.0f * c1, t2, c0);
    const float a = fmaf(c0, g, c1 * t2 * t);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.442695041f * a));
}

// The step of a group of an 8-bit checkpoint from its largest magnitude:
// max / 127 rounded up to bf16, at least 2^-126; NaN where max is not finite.
__device__ __forceinline__ float step8(float top)
{
    const float s = fmaxf(top / 127.0f, 1.17549435e-38f);
    const unsigned up = (__float_as_uint(s) + 0xffffu) & 0xffff0000u;
    return top <= 3.40282347e38f ? __uint_as_float(up) : __uint_as_float(0x7fc00000u);
}

// Four values to int8, with inv = 1 / step; 0 for a NaN step.
__device__ __forceinline__ unsigned pack8x4(float a, float b, float c, float d, float inv)
{
    const auto one = [&](float v) -> unsigned {
        const float q = rintf(v * inv);
        return (unsigned)(int)(q >= -127.0f ? fminf(q, 127.0f) : (q < 0.0f ? -127.0f : 0.0f)) & 0xffu;
    };
    return one(a) | (one(b) << 8) | (one(c) << 16) | (one(d) << 24);
}

__device__ __forceinline__ float int8_of(unsigned u, int i) { return (float)(int)(signed char)(u >> (8 * i)); }

// Tile `t` of the expert segments cut into ceil(count / rows_per_tile) pieces
// each: its expert, or -1 past the last; *first and *count are its rows.
// Every lane of the wave calls it with the same t and gets the same answer.
// The rows of a segment are shared out evenly over its tiles in units of
// `unit` rows (rows_per_tile a multiple of it), so that a segment a little
// longer than one tile does not leave the next one nearly empty.
__device__ __forceinline__ int segment_tile(const int32_t* __restrict__ offset, int E, int rows_per_tile, int unit,
                                            int t, int* first, int* count)
{
    // a lane has `per` neighbouring experts; their offsets are loaded together, and again (from the cache) to find
    // the tile's among them
    const int lane = lane_id(), per = (E + kWave - 1) / kWave, e0 = min(lane * per, E), e1 = min(e0 + per, E);
    const auto tiles_of = [=](int rows) { return (rows + rows_per_tile - 1) / rows_per_tile; };
    int mine = 0, lo = offset[e0];
#pragma unroll 4
    for (int i = 1; i <= per; ++i) {
        const int hi = offset[min(e0 + i, e1)];
        mine += tiles_of(hi - lo);
        lo = hi;
    }
    const int upto = wave_inclusive_scan(mine);
    const unsigned long long m = __ballot(upto > t);
    if (!m) return -1;
    const int src = __builtin_ctzll(m);
    int left = t - (upto - mine), found = 0, at = 0, rows = 0, tiles = 0;
    lo = offset[e0];
#pragma unroll 4
    for (int i = 1; i <= per; ++i) {
        const int hi = offset[min(e0 + i, e1)], n = tiles_of(hi - lo);
        if (left >= 0 && left < n) {
            found = e0 + i - 1;
            at = lo;
            rows = hi - lo;
            tiles = n;
            break;
        }
        left -= n;
        lo = hi;
    }
    const int i = __builtin_amdgcn_readlane(left, src), first_row = __builtin_amdgcn_readlane(at, src);
    const int all = __builtin_amdgcn_readlane(rows, src), n = __builtin_amdgcn_readlane(tiles, src);
    const int units = (all + unit - 1) / unit, each = (units + n - 1) / n * unit;
    *first = first_row + i * each;
    *count = min(each, all - i * each);
    return __builtin_amdgcn_readlane(found, src);
}

}  // namespace ms
