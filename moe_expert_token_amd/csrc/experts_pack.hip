// experts_pack.hip -- 8-bit activation checkpoints of rows: q = rne(x / step), step = max |x| / 127 of 32 neighbours
// rounded up to bf16, so that no quotient passes 127 and q * step is exact in fp32.
#include "experts.h"

namespace ms {
namespace {

// Both kernels are bound by the bytes they move: a lane has one vector of 8 elements, four neighbouring lanes a group
// (two shuffles find its largest), and vectors that nothing reads again soon pass the caches by.  8192 x 7168, 180 MB
// each way: 34 us a kernel, 5.3 TB/s (a plain copy of 2 GiB runs at 6.5).

// The vector of unit i, its group g and whether it is in the row; units are four a group.  Where rows are whole
// groups (Whole) units and vectors are the same, and no division is needed.
template <bool Whole>
__device__ __forceinline__ bool vector_of(int64_t i, int64_t units, int groups, int V, int64_t* at, int64_t* g)
{
    *g = i >> 2;
    *at = i;
    if (Whole) return i < units;
    const int64_t row = *g / groups;
    const int v = 4 * (int)(*g - row * groups) + ((int)i & 3);
    *at = row * V + v;
    return i < units && v < V;
}

// The lanes of a row's last group that lie past its end hold zeros.
template <bool Whole>
__global__ __launch_bounds__(256) void pack8_kernel(const u32x4* __restrict__ x, int64_t units, int groups, int V,
                                                    u32x2* __restrict__ q, unsigned short* __restrict__ scale,
                                                    GridSpan span)
{
    const int64_t i = (int64_t)span_block(span) * 256 + threadIdx.x;
    int64_t at, g;
    const bool ok = vector_of<Whole>(i, units, groups, V, &at, &g);
    u32x4 d = {0, 0, 0, 0};
    if (ok) d = load_row16<true>(x + at);
    float f[8], top = 0;
    bool bad = false;
    for (int c = 0; c < 4; ++c) { f[2 * c] = bf16_lo(d[c]); f[2 * c + 1] = bf16_hi(d[c]); }
    for (int c = 0; c < 8; ++c) { top = fmaxf(top, fabsf(f[c])); bad |= !(fabsf(f[c]) <= 3.40282347e38f); }
    if (bad) top = __uint_as_float(0x7f800000u);
    top = fmaxf(top, __shfl_xor(top, 1, kWave));
    top = fmaxf(top, __shfl_xor(top, 2, kWave));
    const float step = step8(top), inv = 1.0f / step;
    if (!ok) return;
    __builtin_nontemporal_store(u32x2{pack8x4(f[0], f[1], f[2], f[3], inv), pack8x4(f[4], f[5], f[6], f[7], inv)},
                                q + at);
    if ((i & 3) == 0) scale[g] = (unsigned short)(__float_as_uint(step) >> 16);
}

// x' in bf16; one past its range becomes its largest finite value.
__device__ __forceinline__ unsigned value8(unsigned u, int i, float step)
{
    const float v = int8_of(u, i) * step;
    if (v != v) return 0x7fc0u;
    return bf16_rne(fminf(fmaxf(v, -3.38953139e38f), 3.38953139e38f));
}

template <bool Whole>
__global__ __launch_bounds__(256) void unpack8_kernel(const u32x2* __restrict__ q,
                                                      const unsigned short* __restrict__ scale, int64_t units,
                                                      int groups, int V, u32x4* __restrict__ x, GridSpan span)
{
    const int64_t i = (int64_t)span_block(span) * 256 + threadIdx.x;
    int64_t at, g;
    if (!vector_of<Whole>(i, units, groups, V, &at, &g)) return;
    const u32x2 d = __builtin_nontemporal_load(q + at);
    const float step = __uint_as_float((unsigned)scale[g] << 16);
    u32x4 out;
    for (int c = 0; c < 4; ++c)
        out[c] = value8(d[c >> 1], 2 * (c & 1), step) | (value8(d[c >> 1], 2 * (c & 1) + 1, step) << 16);
    store_row16<true>(out, x + at);
}

}  // namespace

hipError_t launch_pack8(const void* x, int64_t rows, int cols, void* q, void* scale, hipStream_t s)
{
    const int groups = (cols + kGroup8 - 1) / kGroup8;
    const int64_t units = rows * groups * 4;
    return launch_spans((units + 255) / 256, 256, [&](dim3 grid, GridSpan span) {
        const auto kernel = cols % kGroup8 ? pack8_kernel<false> : pack8_kernel<true>;
        kernel<<<grid, 256, 0, s>>>((const u32x4*)x, units, groups, cols / 8, (u32x2*)q, (unsigned short*)scale, span);
    });
}

hipError_t launch_unpack8(const void* q, const void* scale, int64_t rows, int cols, void* x, hipStream_t s)
{
    const int groups = (cols + kGroup8 - 1) / kGroup8;
    const int64_t units = rows * groups * 4;
    return launch_spans((units + 255) / 256, 256, [&](dim3 grid, GridSpan span) {
        const auto kernel = cols % kGroup8 ? unpack8_kernel<false> : unpack8_kernel<true>;
        kernel<<<grid, 256, 0, s>>>((const u32x2*)q, (const unsigned short*)scale, units, groups, cols / 8,
                                            (u32x4*)x, span);
    });
}

}  // namespace ms
