// experts_w4.hip -- the experts' block with 4-bit weights, and their making.
#include "experts.h"

namespace ms {
namespace {

// The dot product of one bf16 row with one row of 4-bit weights, over the wave.
__device__ float w4_dot(const unsigned short* x, const unsigned char* q, const unsigned short* sc, int K, int group)
{
    const int lane = lane_id();
    float acc = 0;
    for (int k = 8 * lane; k < K; k += 8 * kWave) {
        const unsigned v = *(const unsigned*)(q + k / 2);
        const u32x4 xs = *(const u32x4*)(x + k);
        float part = 0;
        for (int i = 0; i < 4; ++i) {
            part = fmaf((float)((int)((v >> (8 * i)) & 15) - 8), bf16_lo(xs[i]), part);
            part = fmaf((float)((int)((v >> (8 * i + 4)) & 15) - 8), bf16_hi(xs[i]), part);
        }
        acc = fmaf(part, __uint_as_float((unsigned)sc[k / group] << 16), acc);
    }
    for (int d = 1; d < kWave; d <<= 1) acc += __shfl_xor(acc, d, kWave);
    return acc;
}

constexpr int kFeatures = 64;  // of a block

__global__ __launch_bounds__(256) void w4_up_kernel(ExpertShape S, const unsigned short* xe, const unsigned char* q,
                                                    const unsigned short* sc, int group, unsigned short* h)
{
    if (*S.status) return;
    int r0, nr;
    const int e = segment_tile(S.offset, S.E, 16, 16, blockIdx.x, &r0, &nr);
    if (e < 0) return;
    const int64_t row0 = (int64_t)e * 2 * S.I;
    for (int c = blockIdx.y * kFeatures + wave_id(); c < min(S.I, (int)(blockIdx.y + 1) * kFeatures); c += 4)
        for (int r = r0; r < r0 + nr; ++r) {
            const unsigned short* x = xe + (int64_t)r * S.H;
            const float g = w4_dot(x, q + (row0 + c) * (S.H / 2), sc + (row0 + c) * (S.H / group), S.H, group);
            const float u = w4_dot(x, q + (row0 + S.I + c) * (S.H / 2), sc + (row0 + S.I + c) * (S.H / group), S.H, group);
            float slope;
            const float v = g * gate_sigmoid(g, S.c0, S.c1, &slope) * u;
            if (lane_id() == 0) h[(int64_t)r * S.I + c] = (unsigned short)bf16_rne(v);
        }
}

__global__ __launch_bounds__(256) void w4_down_kernel(ExpertShape S, const unsigned short* h, const unsigned char* q,
                                                      const unsigned short* sc, int group, unsigned short* ye)
{
    if (*S.status) return;
    int r0, nr;
    const int e = segment_tile(S.offset, S.E, 16, 16, blockIdx.x, &r0, &nr);
    if (e < 0) return;
    const int64_t row0 = (int64_t)e * S.H;
    for (int c = blockIdx.y * kFeatures + wave_id(); c < min(S.H, (int)(blockIdx.y + 1) * kFeatures); c += 4)
        for (int r = r0; r < r0 + nr; ++r) {
            const float y = w4_dot(h + (int64_t)r * S.I, q + (row0 + c) * (S.I / 2), sc + (row0 + c) * (S.I / group), S.I, group);
            if (lane_id() == 0) ye[(int64_t)r * S.H + c] = (unsigned short)bf16_rne(y);
        }
}

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

int row_tiles(const ExpertShape& S) { return S.P / 16 + (S.P < S.E ? S.P : S.E); }

}  // namespace

hipError_t launch_w4_up(const ExpertShape& S, const void* xe, const void* q, const void* scale, int group, void* h,
                        hipStream_t s)
{
    w4_up_kernel<<<dim3(row_tiles(S), (S.I + kFeatures - 1) / kFeatures), 256, 0, s>>>(
        S, (const unsigned short*)xe, (const unsigned char*)q, (const unsigned short*)scale, group, (unsigned short*)h);
    return hipGetLastError();
}

hipError_t launch_w4_down(const ExpertShape& S, const void* h, const void* q, const void* scale, int group, void* ye,
                          hipStream_t s)
{
    w4_down_kernel<<<dim3(row_tiles(S), (S.H + kFeatures - 1) / kFeatures), 256, 0, s>>>(
        S, (const unsigned short*)h, (const unsigned char*)q, (const unsigned short*)scale, group, (unsigned short*)ye);
    return hipGetLastError();
}

hipError_t launch_w4_quantize(const void* w, int64_t rows, int cols, int group, void* q, void* scale, hipStream_t s)
{
    const int64_t groups = rows * (cols / group);
    return launch_spans((groups + 255) / 256, 256, [&](dim3 grid, GridSpan span) {
        w4_quantize_kernel<<<grid, 256, 0, s>>>((const unsigned short*)w, groups, group, (unsigned char*)q,
                                                (unsigned short*)scale, span);
    });
}

}  // namespace ms
