// experts_ffn.hip -- the matrix products of the experts' gated block.
#include <type_traits>

#include "experts_gemm.h"

namespace ms {
namespace {

// ---- from accumulators to rows ----

__device__ __forceinline__ u32x2 pack4(f32x4 v) { return u32x2{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3])}; }

__device__ __forceinline__ f32x4 load4(const void* p, int64_t at)
{
    const u32x2 u = *(const u32x2*)((const unsigned short*)p + at);
    return f32x4{bf16_lo(u[0]), bf16_hi(u[0]), bf16_lo(u[1]), bf16_hi(u[1])};
}

// A staged output tile: rows of `Bytes` bytes in LDS, their 16-byte pieces permuted by the row so that the sixteen
// rows a wave writes at once spread over the banks; from there rows go out whole.
template <int Bytes>
struct Stage {
    static __device__ __forceinline__ char* at(char* lds, int row, int byte)
    {
        return lds + row * Bytes + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15);
    }

    // Rows [0, nr) and bytes [0, valid) of the tile to out + row * ld; Vec divides valid and the rows' alignment.
    template <class Vec>
    static __device__ __forceinline__ void store(const char* lds, int nr, int valid, char* out, int64_t ld)
    {
        constexpr int kLanes = Bytes / (int)sizeof(Vec), kRows = kGemmThreads / kLanes;
        const int b = (int)(threadIdx.x % kLanes) * (int)sizeof(Vec);
        if (b >= valid) return;
        for (int r = threadIdx.x / kLanes; r < nr; r += kRows)
            *(Vec*)(out + r * ld + b) = *(const Vec*)at((char*)lds, r, b);
    }
};

// The block's place among `tiles` x `across`: chunks of 32 neighbouring places go to one XCD (blocks are dealt to
// the eight in turn), and within a chunk four row tiles meet eight feature tiles, so its L2 sees each operand
// tile several times at once.
struct Place {
    int tile, across;
};
__device__ __forceinline__ Place place_of(const GridSpan& g, int across)
{
    const int b = span_block(g), slot = b >> 3, i = ((slot >> 5) * 8 + (b & 7)) * 32 + (slot & 31);
    const int group = i / (4 * across), rest = i - group * 4 * across;
    return Place{group * 4 + (rest & 3), rest >> 2};
}

// Blocks that cover tiles x across under place_of.
int64_t places(int64_t tiles, int across) { return ((tiles + 3) / 4 * 4 * across + 255) / 256 * 256; }

// Calls f with the fragment rows (1 .. 8) that cover nr rows as a constant.
template <class F>
__device__ __forceinline__ void with_rows(int nr, F&& f)
{
    switch ((nr + 31) >> 5) {
        case 1: f(std::integral_constant<int, 1>()); break;
        case 2: f(std::integral_constant<int, 2>()); break;
        case 3: f(std::integral_constant<int, 3>()); break;
        case 4: f(std::integral_constant<int, 4>()); break;
        case 5: f(std::integral_constant<int, 5>()); break;
        case 6: f(std::integral_constant<int, 6>()); break;
        case 7: f(std::integral_constant<int, 7>()); break;
        default: f(std::integral_constant<int, 8>()); break;
    }
}

// ---- the kernels ----

// Largest magnitude over the 32 features that the four lanes of a row hold in a and b; infinity if any is not
// finite.  Features past the width (`past`) count as zero.
__device__ __forceinline__ float group_top(f32x4 a, f32x4 b, bool past_a, bool past_b)
{
    float top = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = past_a ? 0.0f : fabsf(a[i]), y = past_b ? 0.0f : fabsf(b[i]);
        top = fmaxf(top, fmaxf(x, y));
        bad |= !(x <= 3.40282347e38f) || !(y <= 3.40282347e38f);
    }
    if (bad) top = __uint_as_float(0x7f800000u);
    top = fmaxf(top, __shfl_xor(top, 16, kWave));
    return fmaxf(top, __shfl_xor(top, 32, kWave));
}

constexpr int kUpFeatures = kTileFeatures / 2;  // of h: each of them takes a gate and an up feature

__global__ __launch_bounds__(kGemmThreads, 2) void ffn_up_kernel(ExpertShape S, const char* xe, const char* w,
                                                                 char* h, SavedActs saved, int across, GridSpan span)
{
    __shared__ __align__(1024) char lds[kGemmLds];
    if (*S.status) return;
    const Place at = place_of(span, across);
    int row0, nr;
    const int e = segment_tile(S.offset, S.E, kTileRows, 32, at.tile, &row0, &nr);
    if (e < 0) return;
    const int c0 = at.across * kUpFeatures, H = S.H, I = S.I;
    KContiguous r, f;
    r.init(xe + (int64_t)row0 * H * 2, H, nr, H);
    // 64 LDS rows are 32 gate rows (loaded by waves 0 .. 3) and the 32 up rows of the same features: one wave's
    const int valid = min(kUpFeatures, I - c0);
    f.init(w + ((int64_t)e * 2 * I + c0 + (wave_id() >= 4 ? I : 0)) * H * 2, H, valid, H, 32, (threadIdx.x >> 3) & 31);
    const int lane = lane_id(), wr = wave_id() >> 2, wf = wave_id() & 3, groups = (I + kGroup8 - 1) / kGroup8;
    with_rows(nr, [&](auto mf) {
        constexpr int MF = decltype(mf)::value;
        Acc<MF> acc;
        tile_product<MF>(r, f, H, lds, acc);
        typedef Stage<kUpFeatures * 2> Wide;
        typedef Stage<kUpFeatures> Narrow;
        char* const second = lds + 256 * kUpFeatures * 2;
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int row = 16 * (MF * wr + m) + (lane & 15);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = 32 * wf + 16 * i + 4 * (lane >> 4);
                f32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float slope;
                    v[j] = acc[m][i][j] * gate_sigmoid(acc[m][i][j], S.c0, S.c1, &slope) * acc[m][2 + i][j];
                }
                *(u32x2*)Wide::at(lds, row, 2 * c) = pack4(v);
                if (saved.data && !saved.scale) *(u32x2*)Wide::at(second, row, 2 * c) = pack4(acc[m][i]);
            }
            if (!saved.scale) continue;
            const int c = 32 * wf + 4 * (lane >> 4);
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const f32x4 a = acc[m][2 * which], b = acc[m][2 * which + 1];
                const float step = step8(group_top(a, b, c0 + c >= I, c0 + c + 16 >= I)), inv = 1.0f / step;
                char* const to = second + which * 256 * kUpFeatures;
                *(unsigned*)Narrow::at(to, row, c) = pack8x4(a[0], a[1], a[2], a[3], inv);
                *(unsigned*)Narrow::at(to, row, c + 16) = pack8x4(b[0], b[1], b[2], b[3], inv);
                if (row < nr && lane < 16 && c0 + 32 * wf < I)
                    ((unsigned short*)saved.scale)[((int64_t)(row0 + row) * 2 + which) * groups + c0 / 32 + wf] =
                        (unsigned short)(__float_as_uint(step) >> 16);
            }
        }
        __syncthreads();
        Wide::store<u32x4>(lds, nr, 2 * valid, h + ((int64_t)row0 * I + c0) * 2, (int64_t)I * 2);
        if (!saved.data) return;
        char* const out = (char*)saved.data + ((int64_t)row0 * 2 * I + c0) * (saved.scale ? 1 : 2);
        if (saved.scale) {
            Narrow::store<u32x2>(second, nr, valid, out, (int64_t)2 * I);
            Narrow::store<u32x2>(second + 256 * kUpFeatures, nr, valid, out + I, (int64_t)2 * I);
            return;
        }
        Wide::store<u32x4>(second, nr, 2 * valid, out, (int64_t)4 * I);
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *(u32x2*)Wide::at(lds, 16 * (MF * wr + m) + (lane & 15), 2 * (32 * wf + 16 * i + 4 * (lane >> 4))) =
                    pack4(acc[m][2 + i]);
        __syncthreads();
        Wide::store<u32x4>(lds, nr, 2 * valid, out + (int64_t)2 * I, (int64_t)4 * I);
    });
}

typedef Stage<kTileFeatures * 2> WideStage;

// The accumulators, put through `value` (m, n, row, feature, acc) -> packed bf16, to rows of `out`.
template <int MF, class Value>
__device__ __forceinline__ void write_tile(char* lds, int nr, int valid, char* out, int64_t ld, Value value)
{
    const int lane = lane_id(), wr = wave_id() >> 2, wf = wave_id() & 3;
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int row = 16 * (MF * wr + m) + (lane & 15), c = 64 * wf + 16 * n + 4 * (lane >> 4);
            *(u32x2*)WideStage::at(lds, row, 2 * c) = value(m, n, row, c);
        }
    __syncthreads();
    WideStage::store<u32x4>(lds, nr, 2 * valid, out, ld);
}

// out[row] = in[row] F^T for the rows of every expert; in [P, K], out [P, N], F of an expert [N][K] (or, Strided,
// [K][N]) at w.
template <bool Strided>
__global__ __launch_bounds__(kGemmThreads, 2) void ffn_rows_kernel(ExpertShape S, const char* in, int K,
                                                                   const char* w, int N, char* out, int across,
                                                                   GridSpan span)
{
    __shared__ __align__(1024) char lds[kGemmLds];
    if (*S.status) return;
    const Place at = place_of(span, across);
    int row0, nr;
    const int e = segment_tile(S.offset, S.E, kTileRows, 32, at.tile, &row0, &nr);
    if (e < 0) return;
    const int n0 = at.across * kTileFeatures;
    KContiguous r;
    r.init(in + (int64_t)row0 * K * 2, K, nr, K);
    typename std::conditional<Strided, KStrided, KContiguous>::type f;
    if constexpr (Strided) f.init(w + ((int64_t)e * K * N + n0) * 2, N, N - n0, K);
    else f.init(w + ((int64_t)e * N + n0) * K * 2, K, min(N - n0, kTileFeatures), K);
    with_rows(nr, [&](auto mf) {
        constexpr int MF = decltype(mf)::value;
        Acc<MF> acc;
        tile_product<MF>(r, f, K, lds, acc);
        write_tile<MF>(lds, nr, min(N - n0, kTileFeatures), out + ((int64_t)row0 * N + n0) * 2, (int64_t)N * 2,
                       [&](int m, int n, int, int) { return pack4(acc[m][n]); });
    });
}

__global__ __launch_bounds__(kGemmThreads, 2) void ffn_dh_kernel(ExpertShape S, const char* gy, const char* w,
                                                                 SavedActs saved, char* h, char* dgu, int across,
                                                                 GridSpan span)
{
    __shared__ __align__(1024) char lds[kGemmLds];
    if (*S.status) return;
    const Place at = place_of(span, across);
    int row0, nr;
    const int e = segment_tile(S.offset, S.E, kTileRows, 32, at.tile, &row0, &nr);
    if (e < 0) return;
    const int n0 = at.across * kTileFeatures, H = S.H, I = S.I, groups = (I + kGroup8 - 1) / kGroup8;
    KContiguous r;
    KStrided f;
    r.init(gy + (int64_t)row0 * H * 2, H, nr, H);
    f.init(w + ((int64_t)e * H * I + n0) * 2, I, I - n0, H);
    const int valid = min(I - n0, kTileFeatures);
    with_rows(nr, [&](auto mf) {
        constexpr int MF = decltype(mf)::value;
        Acc<MF> acc;
        tile_product<MF>(r, f, H, lds, acc);
        // each pass reads the saved pre-activations again (from the caches) rather than hold three tiles
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            char* const out = pass == 0 ? h + ((int64_t)row0 * I + n0) * 2
                                        : dgu + ((int64_t)row0 * 2 * I + (pass == 1 ? 0 : I) + n0) * 2;
            write_tile<MF>(lds, nr, valid, out, (int64_t)I * (pass == 0 ? 2 : 4), [&](int m, int n, int row, int c) {
                f32x4 g = {0, 0, 0, 0}, u = {0, 0, 0, 0};
                if (row < nr && c < valid) {
                    const int64_t at = (int64_t)(row0 + row) * 2 * I + n0 + c;
                    if (saved.scale) {
                        const unsigned short* sc =
                            (const unsigned short*)saved.scale + (int64_t)(row0 + row) * 2 * groups + (n0 + c) / kGroup8;
                        const float sg = __uint_as_float((unsigned)sc[0] << 16);
                        const float su = __uint_as_float((unsigned)sc[groups] << 16);
                        const unsigned qg = *(const unsigned*)((const char*)saved.data + at);
                        const unsigned qu = *(const unsigned*)((const char*)saved.data + at + I);
#pragma unroll
                        for (int j = 0; j < 4; ++j) { g[j] = int8_of(qg, j) * sg; u[j] = int8_of(qu, j) * su; }
                    } else {
                        g = load4(saved.data, at);
                        u = load4(saved.data, at + I);
                    }
                }
                f32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float slope;
                    const float s = gate_sigmoid(g[j], S.c0, S.c1, &slope), a = g[j] * s, d = acc[m][n][j];
                    v[j] = pass == 0 ? a * u[j] : pass == 1 ? d * u[j] * fmaf(a * (1.0f - s), slope, s) : d * a;
                }
                return pack4(v);
            });
            __syncthreads();
        }
    });
}

// out[e] = a^T b over the rows of expert e: both operands' k is the row.
__global__ __launch_bounds__(kGemmThreads, 2) void ffn_wgrad_kernel(ExpertShape S, const char* a, int na,
                                                                    const char* b, int nb, char* out, int down,
                                                                    int across, GridSpan span)
{
    __shared__ __align__(1024) char lds[kGemmLds];
    if (*S.status) return;
    const Place at = place_of(span, across);
    const int e = at.tile / down, m0 = (at.tile - e * down) * kTileRows, n0 = at.across * kTileFeatures;
    if (e >= S.E) return;
    const int q0 = S.offset[e], rows = S.offset[e + 1] - q0;
    KStrided r, f;
    r.init(a + ((int64_t)q0 * na + m0) * 2, na, na - m0, rows);
    f.init(b + ((int64_t)q0 * nb + n0) * 2, nb, nb - n0, rows);
    Acc<8> acc;
    tile_product<8>(r, f, rows, lds, acc);
    write_tile<8>(lds, min(na - m0, kTileRows), min(nb - n0, kTileFeatures),
                  out + (((int64_t)e * na + m0) * nb + n0) * 2, (int64_t)nb * 2,
                  [&](int m, int n, int, int) { return pack4(acc[m][n]); });
}

int64_t row_tiles(const ExpertShape& S) { return (int64_t)S.P / kTileRows + (S.P < S.E ? S.P : S.E); }
int tiles_of(int n, int tile) { return (n + tile - 1) / tile; }

}  // namespace

hipError_t launch_ffn_up(const ExpertShape& S, const void* xe, const void* w_gate_up, void* h, SavedActs saved,
                         hipStream_t s)
{
    const int across = tiles_of(S.I, kUpFeatures);
    return launch_spans(places(row_tiles(S), across), kGemmThreads, [&](dim3 grid, GridSpan span) {
        ffn_up_kernel<<<grid, kGemmThreads, 0, s>>>(S, (const char*)xe, (const char*)w_gate_up, (char*)h, saved, across,
                                                    span);
    });
}

hipError_t launch_ffn_down(const ExpertShape& S, const void* h, const void* w_down, void* ye, hipStream_t s)
{
    const int across = tiles_of(S.H, kTileFeatures);
    return launch_spans(places(row_tiles(S), across), kGemmThreads, [&](dim3 grid, GridSpan span) {
        ffn_rows_kernel<false><<<grid, kGemmThreads, 0, s>>>(S, (const char*)h, S.I, (const char*)w_down, S.H, (char*)ye,
                                                             across, span);
    });
}

hipError_t launch_ffn_dh(const ExpertShape& S, const void* grad_ye, const void* w_down, SavedActs saved, void* h,
                         void* dgu, hipStream_t s)
{
    const int across = tiles_of(S.I, kTileFeatures);
    return launch_spans(places(row_tiles(S), across), kGemmThreads, [&](dim3 grid, GridSpan span) {
        ffn_dh_kernel<<<grid, kGemmThreads, 0, s>>>(S, (const char*)grad_ye, (const char*)w_down, saved, (char*)h,
                                                    (char*)dgu, across, span);
    });
}

hipError_t launch_ffn_dx(const ExpertShape& S, const void* dgu, const void* w_gate_up, void* grad_xe, hipStream_t s)
{
    const int across = tiles_of(S.H, kTileFeatures);
    return launch_spans(places(row_tiles(S), across), kGemmThreads, [&](dim3 grid, GridSpan span) {
        ffn_rows_kernel<true><<<grid, kGemmThreads, 0, s>>>(S, (const char*)dgu, 2 * S.I, (const char*)w_gate_up, S.H,
                                                            (char*)grad_xe, across, span);
    });
}

hipError_t launch_ffn_wgrad(const ExpertShape& S, const void* a, int na, const void* b, int nb, void* out,
                            hipStream_t s)
{
    const int down = tiles_of(na, kTileRows), across = tiles_of(nb, kTileFeatures);
    return launch_spans(places((int64_t)S.E * down, across), kGemmThreads, [&](dim3 grid, GridSpan span) {
        ffn_wgrad_kernel<<<grid, kGemmThreads, 0, s>>>(S, (const char*)a, na, (const char*)b, nb, (char*)out, down,
                                                       across, span);
    });
}

}  // namespace ms
