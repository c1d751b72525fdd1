// experts_w4.hip -- the making of 4-bit weights: step = max |w| / 7 of a group, rounded to bf16, q = rne(w / step) + 8.
// Done once for a set of weights.  Bound by its access: a lane reads a whole group, so a wave's loads lie a group apart.
// 8 experts' [8192][4096]: 245 us with groups of 32 (2.8 TB/s), 1454 with groups of 128 (0.46 TB/s).
#include "experts.h"

namespace ms {
namespace {

// One lane a group.
__global__ __launch_bounds__(256) void w4_quantize_kernel(const unsigned short* __restrict__ w, int64_t groups,
                                                          int group, unsigned char* __restrict__ q,
                                                          unsigned short* __restrict__ scale, GridSpan span)
{
    const int64_t i = (int64_t)span_block(span) * 256 + threadIdx.x;
    if (i >= groups) return;
    const u32x4* p = (const u32x4*)(w + i * group);
    float top = 0;
    bool bad = false;
    for (int j = 0; j < group / 8; ++j) {
        const u32x4 v = p[j];
        for (int c = 0; c < 4; ++c) {
            const float a = fabsf(bf16_lo(v[c])), b = fabsf(bf16_hi(v[c]));
            bad |= !(a <= 3.40282347e38f) || !(b <= 3.40282347e38f);
            top = fmaxf(top, fmaxf(a, b));
        }
    }
    const unsigned sb = bad ? 0x7fc0u : bf16_rne(fmaxf(top / 7.0f, 1.17549435e-38f));
    const float inv = bad ? 0.0f : 1.0f / __uint_as_float(sb << 16);
    scale[i] = (unsigned short)sb;
    const auto one = [&](float v) -> unsigned {
        return bad ? 8u : (unsigned)((int)fminf(fmaxf(rintf(v * inv), -8.0f), 7.0f) + 8);
    };
    for (int j = 0; j < group / 8; ++j) {
        const u32x4 v = p[j];
        unsigned out = 0;
        for (int c = 0; c < 4; ++c) out |= (one(bf16_lo(v[c])) | (one(bf16_hi(v[c])) << 4)) << (8 * c);
        ((unsigned*)(q + i * (group / 2)))[j] = out;
    }
}

}  // namespace

hipError_t launch_w4_quantize(const void* w, int64_t rows, int cols, int group, void* q, void* scale, hipStream_t s)
{
    const int64_t groups = rows * (cols / group);
    return launch_spans((groups + 255) / 256, 256, [&](dim3 grid, GridSpan span) {
        w4_quantize_kernel<<<grid, 256, 0, s>>>((const unsigned short*)w, groups, group, (unsigned char*)q,
                                                (unsigned short*)scale, span);
    });
}

}  // namespace ms
