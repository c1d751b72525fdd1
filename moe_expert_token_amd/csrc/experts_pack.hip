// experts_pack.hip -- 8-bit activation checkpoints of rows.
#include "experts.h"

namespace ms {
namespace {

// One lane a vector of 8 elements; four neighbouring lanes hold a group.  The
// lanes of a row's last group that lie past its end hold zeros.
__global__ __launch_bounds__(256) void pack8_kernel(const u32x4* __restrict__ x, int64_t units, int groups, int V,
                                                    u32x2* __restrict__ q, unsigned short* __restrict__ scale,
                                                    GridSpan span)
{
    const int64_t i = (int64_t)span_block(span) * 256 + threadIdx.x;
    const int64_t g = i >> 2, row = g / groups;
    const int v = 4 * (int)(g - row * groups) + ((int)i & 3);
    const bool ok = i < units && v < V;
    u32x4 d = {0, 0, 0, 0};
    if (ok) d = x[row * V + v];
    float f[8], top = 0;
    bool bad = false;
    for (int c = 0; c < 4; ++c) { f[2 * c] = bf16_lo(d[c]); f[2 * c + 1] = bf16_hi(d[c]); }
    for (int c = 0; c < 8; ++c) { top = fmaxf(top, fabsf(f[c])); bad |= !(fabsf(f[c]) <= 3.40282347e38f); }
    if (bad) top = __uint_as_float(0x7f800000u);
    top = fmaxf(top, __shfl_xor(top, 1, kWave));
    top = fmaxf(top, __shfl_xor(top, 2, kWave));
    const float step = step8(top), inv = 1.0f / step;
    if (!ok) return;
    q[row * V + v] = u32x2{pack8x4(f[0], f[1], f[2], f[3], inv), pack8x4(f[4], f[5], f[6], f[7], inv)};
    if ((i & 3) == 0) scale[g] = (unsigned short)(__float_as_uint(step) >> 16);
}

// x' in bf16; one past its range becomes its largest finite value.
__device__ __forceinline__ unsigned value8(unsigned u, int i, float step)
{
    const float v = int8_of(u, i) * step;
    if (v != v) return 0x7fc0u;
    return bf16_rne(fminf(fmaxf(v, -3.38953139e38f), 3.38953139e38f));
}

__global__ __launch_bounds__(256) void unpack8_kernel(const u32x2* __restrict__ q,
                                                      const unsigned short* __restrict__ scale, int64_t units,
                                                      int groups, int V, u32x4* __restrict__ x, GridSpan span)
{
    const int64_t i = (int64_t)span_block(span) * 256 + threadIdx.x;
    const int64_t g = i >> 2, row = g / groups;
    const int v = 4 * (int)(g - row * groups) + ((int)i & 3);
    if (i >= units || v >= V) return;
    const u32x2 d = q[row * V + v];
    const float step = __uint_as_float((unsigned)scale[g] << 16);
    u32x4 out;
    for (int c = 0; c < 4; ++c)
        out[c] = value8(d[c >> 1], 2 * (c & 1), step) | (value8(d[c >> 1], 2 * (c & 1) + 1, step) << 16);
    x[row * V + v] = out;
}

}  // namespace

hipError_t launch_pack8(const void* x, int64_t rows, int cols, void* q, void* scale, hipStream_t s)
{
    const int groups = (cols + kGroup8 - 1) / kGroup8;
    const int64_t units = rows * groups * 4;
    return launch_spans((units + 255) / 256, 256, [&](dim3 grid, GridSpan span) {
        pack8_kernel<<<grid, 256, 0, s>>>((const u32x4*)x, units, groups, cols / 8, (u32x2*)q, (unsigned short*)scale,
                                          span);
    });
}

hipError_t launch_unpack8(const void* q, const void* scale, int64_t rows, int cols, void* x, hipStream_t s)
{
    const int groups = (cols + kGroup8 - 1) / kGroup8;
    const int64_t units = rows * groups * 4;
    return launch_spans((units + 255) / 256, 256, [&](dim3 grid, GridSpan span) {
        unpack8_kernel<<<grid, 256, 0, s>>>((const u32x2*)q, (const unsigned short*)scale, units, groups, cols / 8,
                                            (u32x4*)x, span);
    });
}

}  // namespace ms
